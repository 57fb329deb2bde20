"""Attention over a 4-bit paged cache against the fp64 reference over the values that it stands for (tolerances as for the
bf16 cache: paged_util.py; the codes' products with bf16 numbers are as exact as bf16's own)."""

import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4, quantise
from paged_util import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def run(fa, b, causal=True, window=0, fill=7.0, **kw):
    o = torch.full((b.T, b.Hq, b.d), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), fill, dtype=torch.float32, device="cuda")
    plan = b.plan(fa, causal=causal, window=window)
    fa.forward_paged4(b.dev["q"], b.cache, plan, out=o, lse=lse, **kw)
    fa.check()
    b.check(o, lse, causal=causal, window=window, fill=fill, scale=kw.get("scale"))
    return o, lse


HEADS = [(1, 1), (4, 2), (8, 1), (6, 2), (16, 1), (5, 5), (14, 2)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_single_tokens(fa, d, Hq, Hkv):
    lens = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 64), (1, 333), (1, 1000)]
    run(fa, Batch4(fa, lens, Hq, Hkv, d, 16, seed=d + Hq, lead=2, pad=3))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_and_strides(fa, d, page):
    lens = [(1, 1), (3, 700), (0, 50), (2, 255), (1, 257), (0, 0)]
    run(fa, Batch4(fa, lens, 4, 2, d, page, seed=page, apart=True))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (True, 200)])
@pytest.mark.parametrize("Hq,Hkv,ql", [(4, 2, 2), (4, 1, 4), (8, 1, 4), (3, 1, 9), (4, 4, 30)])
def test_drafted_tokens(fa, d, causal, window, Hq, Hkv, ql):
    lens = [(ql, ql), (ql, ql + 1), (1, 90), (ql, 500), (0, 3), (max(1, ql - 1), 129)]
    run(fa, Batch4(fa, lens, Hq, Hkv, d, 32, seed=ql, pad=1), causal, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 77)])
@pytest.mark.parametrize("Hq,Hkv,page", [(8, 2, 16), (3, 3, 64), (5, 1, 256)])
def test_chunks(fa, d, causal, window, Hq, Hkv, page):
    lens = [(100, 100), (1, 400), (257, 300), (40, 700), (33, 33)]
    run(fa, Batch4(fa, lens, Hq, Hkv, d, page, seed=page + d), causal, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150)])
def test_chunks_have_the_bits_of_a_bf16_cache(fa, d, causal, window):
    b = Batch4(fa, [(300, 300), (65, 900), (128, 128), (200, 1500)], 8, 2, d, 32, seed=3)
    plan = b.plan(fa, causal=causal, window=window)
    o, lse = fa.forward_paged4(b.dev["q"], b.cache, plan)
    kc, vc = (torch.nan_to_num(x, nan=0.0) for x in (b.kc, b.vc))
    o2, lse2 = fa.forward_paged(b.dev["q"], kc, vc, plan)
    fa.check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_sequence_is_shared(fa, d):
    """Few sequences: their tiles are split among CTAs, and joined by a kernel of its own or by the last CTA."""
    for Hq, Hkv, n in ((8, 1, 20000), (4, 4, 5000), (32, 8, 3001)):
        run(fa, Batch4(fa, [(1, n)], Hq, Hkv, d, 64, seed=n))
    run(fa, Batch4(fa, [(4, 9000), (1, 7)], 8, 1, d, 16, seed=5))


@pytest.mark.parametrize("d", [64, 128])
def test_scale_strided_queries_and_repeats(fa, d):
    b = Batch4(fa, [(1, 200), (2, 100), (1, 40)], 8, 2, d, 16, seed=11)
    big = torch.zeros(b.T, b.Hq + 3, d, dtype=torch.bfloat16, device="cuda")
    big[:, :b.Hq] = b.dev["q"]
    b.dev["q"] = big[:, :b.Hq]
    first = run(fa, b, scale=0.37)
    for _ in range(3):
        again = run(fa, b, scale=0.37)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("ql", [1, 70])
def test_nan_in_a_seen_group_reaches_its_rows(fa, ql):
    b = Batch4(fa, [(ql, 400), (ql, 300)], 4, 2, 128, 16, seed=2)
    page, slot = int(b.table[0, 3]), 5
    b.cache.k_scale[page, 1, slot, 2] = float("nan")
    o, lse = fa.forward_paged4(b.dev["q"], b.cache, b.plan(fa))
    fa.check()
    assert o[:ql, 2:].isnan().all() and lse[:ql, 2:].isnan().all()
    assert not o[:ql, :2].isnan().any() and not o[ql:].isnan().any()


@pytest.mark.parametrize("d", [64, 128])
def test_many_heads_per_kv_head_and_many_sequences(fa, d):
    run(fa, Batch4(fa, [(1, 70), (2, 33)], 130, 1, d, 16, seed=1))
    r = torch.Generator().manual_seed(5)
    lens = [(int(a), int(a) + int(n)) for a, n in zip(torch.randint(0, 3, (700,), generator=r), torch.randint(0, 60, (700,), generator=r))]
    run(fa, Batch4(fa, lens, 2, 1, d, 16, seed=2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 500])
def test_chunks_beside_single_tokens(fa, d, window):
    """Both kinds of tiles at once, the pairs shared by several CTAs and joined behind the small tiles."""
    lens = [(1, 700), (90, 3000), (1, 2000)] + [(1, 40 + 13 * i) for i in range(30)] + [(150, 150), (2, 1500)]
    run(fa, Batch4(fa, lens, 4, 2, d, 64, seed=d + window, lead=1, pad=2), True, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 900)])
def test_chunks_under_a_table_for_long_contexts(fa, d, causal, window):
    """Blocks in the turned order, as for codes that do not fit L2."""
    page, Hkv = 256, 2
    cols = (100 << 20) // (page * Hkv * 2 * (d // 2 + d // 16)) + 1
    lens = [(70, 5000), (1, 300), (260, 1500), (40, 40)]
    run(fa, Batch4(fa, lens, 4, Hkv, d, page, seed=d, extra_cols=cols), causal, window)


@pytest.mark.parametrize("ql", [4, 40])
def test_more_new_tokens_than_cached_ones(fa, ql):
    """The first of them stand before the sequence and see nothing."""
    run(fa, Batch4(fa, [(ql, ql - 2), (1, 50)], 4, 2, 64, 16, seed=ql))


def test_pages_beyond_four_gigabytes(fa):
    Hkv, page, d = 8, 64, 128
    b = Batch4(fa, [(1, 500), (20, 300)], 16, Hkv, d, page, seed=3)
    pages = (1 << 32) // (Hkv * page * d // 2) + 40  # the last ones begin beyond 2^32 bytes of codes
    big = fa.PagedCache4.empty(pages, Hkv, page, d)
    shift = pages - b.num_pages
    for x, y in zip((big.k, big.v, big.k_scale, big.v_scale), (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)):
        x[shift:] = y
    small = run(fa, b)
    lse = small[1]
    w = torch.rand(b.num_pages, Hkv, page, device="cuda")
    want = fa.paged_weights(b.dev["q"], lse, b.cache, w, b.plan(fa), out=torch.zeros_like(w))
    for i, (_, n) in enumerate(b.lens):
        b.dev["table"][i, :(n + page - 1) // page] += shift
    plan = b.plan(fa)
    o, lse2 = fa.forward_paged4(b.dev["q"], big, plan)
    wb = torch.zeros(pages, Hkv, page, device="cuda")
    wb[shift:] = w
    got = fa.paged_weights(b.dev["q"], lse, big, wb, plan, out=torch.zeros_like(wb))
    x = torch.randn(21, 2 * Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    fa.paged_append4(None, x[:, :Hkv], x[:, Hkv:], big, plan)
    fa.check()
    assert torch.equal(o, small[0]) and torch.equal(lse2, lse) and torch.equal(got[shift:], want)
    last = int(b.dev["table"][0, 7])
    _, s, _ = quantise(f64(x[0, :Hkv]))
    assert torch.equal(big.k_scale[last, :, 499 % page].cpu().double(), torch.from_numpy(s))
