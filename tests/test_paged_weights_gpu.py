"""The weight that cached tokens receive, against 64 bits, over a bf16 and a 4-bit cache.

Tolerance: a score is off by e_s = 2 d 2^-24 scale sum|q k|; scale and log2(e) are applied in fp32 (three roundings of the
exponent, whose parts are at most |x| + |lse|), exp2 adds 2^-22: a weight is off by p (e_s + 4 (|x| + |lse|) 2^-24 + 2^-21).
Sums of n rows are fp32 in a fixed order: at most n 2^-24 of the sum; adding the old weight rounds once more.
"""

import math

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4
from paged_util import Batch, assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def reference(b, lse, old, causal, window, scale):
    """(out, tolerance, written) [pages, Hkv, page] of the batch."""
    out, tol, written = old.copy(), np.zeros_like(old), np.zeros(old.shape, dtype=bool)
    G = b.Hq // b.Hkv
    for i, (ql, n) in enumerate(b.lens):
        q, K, z = f64(b.q)[b.cu[i]:b.cu[i] + ql], f64(b.K[i]), f64(lse)[b.cu[i]:b.cu[i] + ql]
        pos = np.arange(n - ql, n)
        t = np.arange(n)
        seen = np.ones((ql, n), dtype=bool)
        if causal or window:
            seen &= t <= pos[:, None]
        if window:
            seen &= t > pos[:, None] - window
        for h in range(b.Hkv):
            total, err = np.zeros(n), np.zeros(n)
            for hq in range(h * G, (h + 1) * G):
                x = scale * (q[:, hq] @ K[:, h].T)
                es = 2 * b.d * 2.0 ** -24 * scale * (np.abs(q[:, hq]) @ np.abs(K[:, h]).T)
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(seen & ~np.isneginf(z[:, hq])[:, None], np.exp(x - z[:, hq, None]), 0)
                    rel = es + 4 * (np.abs(x) + np.abs(np.nan_to_num(z[:, hq, None], neginf=0))) * 2.0 ** -24 + 2.0 ** -21
                total += p.sum(0)
                err += (p * rel).sum(0)
            for k in np.nonzero(seen.any(0))[0] if ql else []:
                at = (int(b.table[i, k // b.page]), h, k % b.page)
                was = 0 if k >= n - ql else old[at]
                out[at] = was + total[k]
                tol[at] = err[k] + (ql * G + 2) * 2.0 ** -24 * abs(out[at])
                written[at] = True
    return out, tol, written


def run(fa, b, four, causal=True, window=0, scale=None, inplace=False, poke=None):
    sc = scale or 1 / math.sqrt(b.d)
    plan = b.plan(fa, causal=causal, window=window)
    if four:
        _, lse = fa.forward_paged4(b.dev["q"], b.cache, plan, scale=scale)
    else:
        _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, scale=scale)
    if poke is not None:
        poke(lse)
    g = torch.Generator().manual_seed(1)
    old = torch.rand(b.num_pages, b.Hkv, b.page, generator=g)
    w = old.cuda()
    out = w if inplace else torch.full_like(w, 7.0)
    got = fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan, scale=scale, out=None if inplace else out)
    fa.check()
    assert got is out
    ref, tol, written = reference(b, lse, f64(old), causal or window > 0, window, sc)
    if not inplace:
        ref[~written] = 7
        assert torch.equal(w.cpu(), old)
    assert_within(out, ref, tol, "weights")
    return out


def make(fa, four, *a, **kw):
    return Batch4(fa, *a, **kw) if four else Batch(*a, **kw)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 1), (14, 2), (3, 3), (17, 1)])
def test_single_tokens(fa, four, d, Hq, Hkv):
    lens = [(1, 1), (1, 15), (1, 16), (0, 40), (1, 129), (0, 0), (1, 700)]
    run(fa, make(fa, four, lens, Hq, Hkv, d, 16, seed=d + Hq, lead=2, pad=3), four)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (64, 256)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50)])
def test_several_tokens(fa, four, d, page, causal, window):
    lens = [(5, 5), (2, 300), (1, 77), (40, 40), (33, 500), (150, 200)]
    run(fa, make(fa, four, lens, 6, 2, d, page, seed=page, pad=1), four, causal, window)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(64, 1), (65, 1), (130, 2), (200, 1)])
def test_many_heads_per_kv_head(fa, four, d, Hq, Hkv):
    """Rows that fill the queries' buffer, and more: they are copied anew for each block."""
    run(fa, make(fa, four, [(1, 300), (0, 5), (1, 1), (2, 140)], Hq, Hkv, d, 32, seed=Hq), four)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 30), (True, 300)])
def test_chunks_beside_single_tokens(fa, four, causal, window):
    lens = [(1, 900), (70, 400), (1, 1), (1, 33), (130, 130), (3, 257), (20, 1000)]
    run(fa, make(fa, four, lens, 4, 2, 128, 16, seed=9, lead=1), four, causal, window)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_many_sequences_in_place_or_not(fa, four, inplace):
    r = np.random.RandomState(3)
    lens = [(int(r.randint(0, 4)), int(r.randint(4, 90))) for _ in range(150)]
    run(fa, make(fa, four, lens, 4, 2, 64, 16, seed=4), four, inplace=inplace)


def test_weights_of_a_step_sum_to_its_rows_and_repeat(fa):
    b = Batch([(1, 5000), (3, 100)], 8, 2, 128, 32, seed=8)
    one, two = run(fa, b, False), run(fa, b, False)
    assert torch.equal(one, two)
    plan = b.plan(fa)
    _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    w = torch.zeros(b.num_pages, 2, 32, device="cuda")
    fa.paged_weights(b.dev["q"], lse, b.kc, w, plan)
    fa.check()
    # Every row's weights sum to 1: 4 tokens of 8 heads. (Each weight off by 2^-19 or so: |x|, |lse| < 16.)
    assert abs(float(w.double().sum()) - 32) < 32 * 2.0 ** -17


@pytest.mark.parametrize("four", [False, True])
def test_rows_that_see_nothing_and_nan(fa, four):
    b = make(fa, four, [(2, 60), (1, 40)], 4, 2, 64, 16, seed=6)

    def poke(lse):
        lse[0, 1] = -math.inf

    run(fa, b, four, poke=poke)
    plan = b.plan(fa)
    w = torch.zeros(b.num_pages, 2, 16, device="cuda")
    lse = torch.zeros(3, 4, device="cuda")
    lse[2, 0] = math.nan
    fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan)
    fa.check()
    ids = b.table[1, :3].long()
    assert w[ids[:2], 0].isnan().all() and w[ids[2], 0, :8].isnan().all() and not w[ids[2], 0, 8:].isnan().any()
    assert not w[:, 1].isnan().any() and not w[b.table[0, :4].long()].isnan().any()


def test_shared_pages_add_up_in_place(fa):
    b = Batch([(1, 64), (1, 64)], 2, 2, 64, 16, seed=7)
    b.dev["table"][1, :3] = b.dev["table"][0, :3]  # a prefix of 48 tokens
    plan = b.plan(fa)
    _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    w = torch.zeros(b.num_pages, 2, 16, device="cuda")
    fa.paged_weights(b.dev["q"], lse, b.kc, w, plan)
    fa.check()
    assert abs(float(w.double().sum()) - 4) < 4 * 2.0 ** -17


def test_strides_and_a_page_out_of_range(fa):
    b = Batch([(1, 50), (2, 40)], 4, 2, 128, 16, seed=5, layout="pshd")
    plan = b.plan(fa)
    _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    old = torch.rand(2, b.num_pages, 24, device="cuda")[:, :, :16].transpose(0, 1)
    out = torch.full((b.num_pages, 3, 16), 7.0, device="cuda")[:, :2]
    q = torch.zeros(3, 4, 136, dtype=torch.bfloat16, device="cuda")
    q[..., :128] = b.dev["q"]
    fa.paged_weights(q[..., :128], lse, b.kc, old, plan, out=out)
    fa.check()
    ref, tol, written = reference(b, lse, f64(old), True, 0, 1 / math.sqrt(128))
    ref[~written] = 7
    assert_within(out, ref, tol, "strided")
    b.dev["table"][0, 1] = b.num_pages + 3
    out.fill_(7.0)
    fa.paged_weights(q[..., :128], lse, b.kc, old, plan, out=out)
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    gone = int(b.table[0, 1])
    written[gone] = False
    ref[gone] = 7
    assert_within(out, ref, tol, "without the page")
