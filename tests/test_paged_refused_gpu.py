"""Sequences that fa_paged_plan refuses leave the others of their batch as they would be without them.

A refused sequence stands first, in the middle or last; the append's cache and queries and the attention's outputs of
all the others are compared with fp64, and nothing of a refused one is written.
"""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch, assert_within, attention_ref, f64, rope_ref, rotary

pytestmark = pytest.mark.gpu

FILL = -7.0
LENS = [(1, 30), (2, 17), (1, 1), (0, 9), (40, 60), (3, 33), (1, 64), (5, 5)]


def _reported(fa, call):
    out = call()
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    fa.check()
    return out


def _check(b, refused, sample=None):
    fa = fa_mod()
    d = b.d
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(b.T, b.Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    inv = rotary(d)
    q_out = torch.full((b.T, b.Hq, d), FILL, dtype=torch.bfloat16, device="cuda")
    o = torch.full((b.T, b.Hq, d), FILL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    before = b.kc.clone(), b.vc.clone()

    plan = _reported(fa, lambda: b.plan(fa))
    fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, out=o, lse=lse)
    fa.paged_append(b.dev["q"], k.cuda(), v.cuda(), b.kc, b.vc, plan, fa.Rotary(inv.cuda()), q_out=q_out)
    fa.check()

    want_k, want_v = (f64(t) for t in before)
    tol_k = np.zeros_like(want_k)
    want_q, tol_q = np.full((b.T, b.Hq, d), FILL), np.zeros((b.T, b.Hq, d))
    mine = np.zeros(b.T, dtype=bool)
    for i, (ql, n) in enumerate(b.lens):
        if i in refused:
            continue
        a = b.cu[i]
        mine[a:a + ql] = True
        for j in range(ql):
            pos = n - ql + j
            p = np.full(d // 2, float(pos))
            want_q[a + j], tol_q[a + j] = rope_ref(f64(b.q[a + j]), p, inv)
            at = int(b.table[i, pos // b.page]), slice(None), pos % b.page
            want_k[at], tol_k[at] = rope_ref(f64(k[a + j]), p, inv)
            want_v[at] = f64(v[a + j])
        if sample is None or i in sample:
            ro, rl, to, tl = attention_ref(f64(b.q[a:a + ql]), f64(b.K[i]), f64(b.V[i]), n, True, 0, d ** -0.5, b.max_q)
            assert_within(o[a:a + ql], ro, to, f"o of sequence {i}")
            assert_within(lse[a:a + ql], rl, tl, f"lse of sequence {i}")
    assert_within(q_out, want_q, tol_q, "rotated queries")
    assert_within(b.kc, want_k, tol_k, "k cache")
    assert_within(b.vc, want_v, 0.0, "v cache")
    assert np.all(f64(o)[~mine] == FILL) and np.all(f64(lse)[~mine] == FILL)
    assert np.all(f64(o)[mine] != FILL)


@pytest.mark.parametrize("value", [-1, 10 ** 6])
@pytest.mark.parametrize("at", [(0,), (1,), (3,), (4,), (6,), (7,), (0, 1), (2, 5), (6, 7)])
@pytest.mark.parametrize("d", [64, 128])
def test_cached_length_out_of_range(value, at, d):
    b = Batch(LENS, 4, 2, d, 16, seed=31, pad=2, lead=1)
    for i in at:
        b.dev["kv_lens"][i] = value
    _check(b, at)


@pytest.mark.parametrize("at", [1, 2, 4, 5, 7])
@pytest.mark.parametrize("value", [-3, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_start_out_of_range(at, value):
    # A start is also the end before it: both sequences are out of range.
    b = Batch(LENS, 4, 2, 64, 16, seed=32, pad=2, lead=1)
    b.dev["cu_q"][at] = value
    _check(b, (at - 1, at))


@pytest.mark.parametrize("at,value", [(2, 0), (5, 2), (6, 4), (7, 1)])
def test_starts_that_fall_back(at, value):
    # The sequence before ends ahead of its start; the one after begins among the tokens of others.
    b = Batch(LENS, 4, 2, 64, 16, seed=33, pad=2, lead=1)
    b.dev["cu_q"][at] = value
    b.max_q = b.T
    _check(b, (at - 1, at))


def test_more_new_tokens_than_promised():
    b = Batch(LENS, 4, 2, 64, 16, seed=34)
    b.max_q = 4
    _check(b, (4, 7))


@pytest.mark.parametrize("at", [(5,), (1023,), (1024,), (0, 700, 1023, 1024, 1499)])
def test_many_sequences(at):
    # More sequences than the plan's kernel has threads.
    r = np.random.default_rng(5)
    b = Batch([(int(r.integers(0, 3)), int(r.integers(2, 40))) for _ in range(1500)], 2, 1, 64, 16, seed=35)
    for i in at:
        b.dev["kv_lens"][i] = -1
    _check(b, at, sample=set(range(0, 1500, 50)) | {x + y for x in at for y in (-1, 1)})


def test_bounds_fall_between_rounds():
    # The fall stands where the plan's threads go on to their next 1024 sequences.
    b = Batch([(1, 20)] * 1100, 2, 1, 64, 16, seed=36)
    b.dev["cu_q"][1024] = 1000
    b.max_q = 100
    # Sequence 1023 ends before its start; 1024 begins among the tokens of others.
    _check(b, (1023, 1024), sample={0, 1000, 1022, 1025, 1099})
