"""Weights in place where a sequence sees tokens that are new in another sequence of the same step: such a slot starts from 0
and holds what all of them give it. (Tolerances: test_paged_weights_gpu.py; sums of several sequences are rounded once per
sequence.)"""

import copy
import math

import pytest
import torch

from gpu_util import fa_mod
from paged_util import assert_within, f64
from test_paged_weights_gpu import make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("writer", [0, 2, 7])
@pytest.mark.parametrize("ql", [1, 9, 600])
def test_tokens_that_are_new_in_another_sequence(fa, four, d, writer, ql):
    page, S, n = 16, 8, 608
    lens = [(1, n + 5 * i + 1) for i in range(S)]
    lens[writer] = (ql, n)
    b = make(fa, four, lens, 4, 2, d, page, seed=ql + writer)
    for i in range(S):  # the writer's 38 pages begin every sequence
        b.table[i, :n // page] = b.table[writer, :n // page]
        b.K[i][:n] = b.K[writer]
    b.dev["table"].copy_(b.table)
    plan = b.plan(fa)
    lse = (6 + torch.randn(b.T, 4, generator=torch.Generator().manual_seed(1))).cuda()
    old = torch.rand(b.num_pages, 2, page, generator=torch.Generator().manual_seed(2))
    ref, tol = f64(old), 0
    for i, (q, m) in enumerate(lens):  # slots of new tokens start from 0
        for x in range(m - q, m):
            ref[int(b.table[i, x // page]), :, x % page] = 0
    for i in range(S):
        one = copy.copy(b)
        one.lens = [(q if j == i else 0, m) for j, (q, m) in enumerate(lens)]
        got, t, _ = reference(one, lse, 0 * ref, True, 0, 1 / math.sqrt(d))
        ref = ref + got
        tol = tol + t
    tol = tol + S * 2.0 ** -24 * abs(ref)
    for _ in range(3):
        w = old.cuda()
        fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan)
        fa.check()
        assert_within(w, ref, tol, "weights")
