"""Queries with lse = -inf give no weight, whatever they hold, and the rows that fill up a tile of 8 give none either: over
keys that every row sees and over those that only some see. (Tolerances: test_paged_weights_gpu.py.)"""

import math

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch, assert_within, f64
from test_paged_weights_gpu import make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def add(fa, b, plan, lse, four, inplace):
    old = torch.rand(b.num_pages, b.Hkv, b.page, generator=torch.Generator().manual_seed(1))
    w = old.cuda()
    out = w if inplace else w.clone()
    fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan, out=out)
    fa.check()
    return f64(old), out


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal,window,inplace", [(True, 0, False), (True, 0, True), (False, 0, False), (True, 300, False)])
def test_shut_out_queries_of_any_value(fa, four, d, value, causal, window, inplace):
    lens = [(2, 700), (1, 300), (40, 500), (130, 900), (1, 1)]  # up to 64 rows, and more
    b = make(fa, four, lens, 8, 2, d, 16, seed=d, lead=1, pad=1)
    plan = b.plan(fa, causal=causal, window=window)
    if four:
        _, lse = fa.forward_paged4(b.dev["q"], b.cache, plan)
    else:
        _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    for tok, head in ((b.cu[0], 0), (b.cu[0] + 1, 7), (b.cu[1], 3), (b.cu[2] + 5, 2), (b.cu[2] + 39, 4), (b.cu[3], 1),
                      (b.cu[3] + 64, 6), (b.cu[3] + 129, 5)):
        lse[tok, head] = -math.inf
        b.dev["q"][tok, head] = value
    old, out = add(fa, b, plan, lse, four, inplace)
    ref, tol, _ = reference(b, lse, old, causal, window, 1 / math.sqrt(d))  # (over the finite queries, at weight 0)
    assert_within(out, ref, tol, "weights")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("ql", [1, 3])
def test_an_infinite_key_under_few_rows(fa, d, G, ql):
    """Its score is -inf for every query: it receives nothing, although the rows that fill up the tile are zeros."""
    b = Batch([(ql, 600), (ql, 250)], 2 * G, 2, d, 16, seed=d + G)
    b.q[:, :, 0] = -b.q[:, :, 0].abs() - 0.5
    b.dev["q"] = b.q.cuda()
    places = [(0, 130), (0, 597 - ql), (1, 17)]
    for i, x in places:
        b.kc[int(b.table[i, x // 16]), :, x % 16, 0] = math.inf
    plan = b.plan(fa)
    _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    for i, x in places:
        b.K[i][x, :, 1:] = 0  # any finite key, for the reference
        b.K[i][x, :, 0] = 2e4  # 2e4 * -0.5 / sqrt(128): a weight of 0 in 64 bits too
    old, out = add(fa, b, plan, lse, False, False)
    assert np.isfinite(f64(lse)).all()
    ref, tol, _ = reference(b, lse, old, True, 0, 1 / math.sqrt(d))
    assert_within(out, ref, tol, "weights")
    for i, x in places:
        at = int(b.table[i, x // 16]), slice(None), x % 16
        np.testing.assert_array_equal(f64(out)[at], old[at])
