"""Attention over a paged cache (fa_paged_plan, fa_fwd_paged) against an fp64 reference.

Slots of the cache past a sequence hold NaN and infinities and unused table entries numbers out of range, so that
whatever is read past a sequence shows. (Before its window: test_paged_unseen_gpu.py.)
"""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch, assert_within, attention_ref, f64

pytestmark = pytest.mark.gpu

FILL = -7.0


def _run(b, causal=True, window=0, scale=None):
    fa = fa_mod()
    o = torch.full((b.T, b.Hq, b.d), FILL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    plan = b.plan(fa, causal, window)
    fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, scale=scale, out=o, lse=lse)
    fa.check()
    b.check(o, lse, causal, window, scale, FILL)
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_single_tokens(d, page):
    _run(Batch([(1, n) for n in (1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 200, 511, 700)], 8, 2, d, page, seed=d + page))


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (6, 2), (5, 1), (14, 2), (16, 1), (20, 1), (34, 2), (130, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_groups(heads, d):
    _run(Batch([(1, 77), (3, 130), (0, 50), (9, 9), (1, 300)], *heads, d, 16, seed=sum(heads)))


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 7), (False, 64), (True, 100),
                                           (True, 5000)])
@pytest.mark.parametrize("d", [64, 128])
def test_masks_over_chunks(causal, window, d):
    _run(Batch([(33, 33), (1, 400), (70, 333), (5, 128), (129, 130), (0, 0), (17, 640)], 4, 2, d, 32, seed=window + d),
         causal, window)


@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 0)], [(4, 2)], [(0, 5), (0, 0)], [(3, 0), (2, 40), (40, 3)],
                                  [(1, 1)] * 70, [(0, 3)] * 40 + [(2, 9)] + [(0, 0)] * 40 + [(1, 30)]])
@pytest.mark.parametrize("window", [0, 3])
def test_short_empty_and_missing_keys(lens, window):
    # Queries before the first cached key see nothing: o = 0 and lse = -inf.
    _run(Batch(lens, 4, 2, 64, 16, seed=len(lens), pad=5, lead=3), True, window)


@pytest.mark.parametrize("lens", [[(257, 257)], [(256, 1000)], [(300, 2500), (1, 1800), (65, 65)], [(600, 601)]])
@pytest.mark.parametrize("heads", [(4, 1), (3, 1), (2, 2)])
def test_long_chunks(lens, heads):
    _run(Batch(lens, *heads, 128, 64, seed=lens[0][0]))
    _run(Batch(lens, *heads, 64, 16, seed=lens[0][0]), window=200)


@pytest.mark.parametrize("keys", [1, 128, 129, 256, 257, 384, 700, 1500])
@pytest.mark.parametrize("new", [9, 20, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_of_one_tile(keys, new, d):
    # At most 128 rows: both halves of the pairs' kernel take every other key block; one block, odd and even counts.
    _run(Batch([(min(new, keys), keys)], 8, 2, d, 16, seed=keys + new))
    _run(Batch([(min(new, keys), keys), (1, 300), (min(new, keys), 2 * keys)], 4, 1, d, 64, seed=keys), window=150)


@pytest.mark.parametrize("heads", [(4, 1), (8, 8), (6, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_and_two_tiles_and_single_tokens_in_one_batch(heads, d):
    r = np.random.default_rng(heads[0] + d)
    lens = [(1, int(r.integers(1, 900))) for _ in range(20)] + [(150, 400), (1, 0), (0, 70), (40, 1000), (300, 333),
                                                               (2, 5), (33, 33)]
    b = Batch([lens[i] for i in r.permutation(len(lens))], *heads, d, 32, seed=6, pad=2)
    o, lse = _run(b)
    o2, lse2 = _run(b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("d", [64, 128])
def test_drafted_tokens(new, d):
    # 8 to 36 rows per kv head: 16-row tiles, 32-row tiles with any part of the second half, and pairs.
    r = np.random.default_rng(new)
    lens = [(int(r.integers(1, new + 1)), int(r.integers(new, 1200))) for _ in range(12)] + [(new, 3000), (new, new)]
    _run(Batch(lens, 8, 2, d, 16, seed=new), window=0)
    _run(Batch(lens, 12, 3, d, 64, seed=new + 50), window=700)
    _run(Batch(lens, 4, 1, d, 128, seed=new + 90), causal=False)
    _run(Batch(lens, 4, 1, d, 32, seed=new + 90), causal=False, window=90)


@pytest.mark.parametrize("lens", [[(1, 400)] * 40 + [(40, 41)], [(300, 300)] * 7 + [(1, 2)], [(1, 3000), (70, 70)],
                                  [(0, 5)] * 3 + [(64, 700)] * 20 + [(2, 90)] * 20, [(90, 300), (0, 7)]])
@pytest.mark.parametrize("heads", [(8, 2), (7, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_beside_chunks(lens, heads, d):
    # Both kinds of tiles at once, from nearly all SMs for the one to nearly all for the other.
    b = Batch(lens, *heads, d, 32, seed=len(lens), pad=1)
    o, lse = _run(b)
    o2, lse2 = _run(b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 8, 16, 32, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("offset", [0, 8])
def test_outputs_of_any_group_and_alignment(G, d, offset):
    # Rows of o leave in boxes, or 32 or 16 bytes at a time: chunks that end inside a warp's rows, o 16 bytes off.
    fa = fa_mod()
    b = Batch([(131, 131), (70, 333), (0, 9), (33, 40), (1, 100)], 2 * G, 2, d, 32, seed=G, pad=3, lead=1)
    o = torch.full((b.T * b.Hq * d + offset,), FILL, dtype=torch.bfloat16, device="cuda")[offset:].view(b.T, b.Hq, d)
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa), out=o, lse=lse)
    fa.check()
    b.check(o, lse, fill=FILL)


@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 9000), (1, 30)], [(2, 7000), (1, 1), (0, 5), (3, 0), (1, 2500)],
                                  [(60, 800), (1, 9000), (2, 3)], [(1, 100)], [(0, 40)]])
@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 2), (32, 1), (130, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_few_tiles_over_all_ctas(lens, heads, d):
    # One to a few tiles with up to all CTAs' partial results each, joined by a kernel of their own; the same bits
    # each time.
    b = Batch(lens, *heads, d, 64, seed=len(lens) + heads[0], pad=2)
    o, lse = _run(b)
    o2, lse2 = _run(b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _run(b, window=2100)


def test_few_tiles_with_nan_infinities_and_masked_starts():
    # A NaN in a visible key makes its head's rows NaN through the join; rows before the first key stay empty.
    fa = fa_mod()
    b = Batch([(4, 6000), (6, 3)], 8, 2, 128, 32)
    page, slot = int(b.table[0, 5990 // 32]), 5990 % 32
    b.kc[page, 0, slot] = float("nan")
    plan = b.plan(fa)
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    fa.check()
    assert torch.isnan(o[:4, :4].float()).all() and torch.isnan(lse[:4, :4]).all()
    b.K[0][5990, 0] = 0
    for h in (slice(4, 8), slice(0, 8)):
        rows = slice(0, 4) if h.start else slice(4, 10)
        i = 0 if h.start else 1
        ro, rl, to, tl = attention_ref(f64(b.q[rows]), f64(b.K[i]), f64(b.V[i]), b.lens[i][1], True, 0, 128 ** -0.5,
                                       max_q=b.max_q)
        assert_within(o[rows, h], ro[:, h], to[:, h], "o")
        assert_within(lse[rows, h], rl[:, h], tl[:, h], "lse")


@pytest.mark.parametrize("layout", ["pshd", "both"])
@pytest.mark.parametrize("lens", [[(1, 100), (1, 333)], [(90, 300), (1, 77)], [(7, 100), (5, 333), (1, 40)]])
def test_cache_layouts_and_strided_queries(layout, lens):
    fa = fa_mod()
    b = Batch(lens, 8, 2, 128, 32, seed=5, layout=layout)
    wide = torch.full((b.T, b.Hq + 3, b.d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1:1 + b.Hq, :b.d]
    q.copy_(b.dev["q"])
    o, lse = fa.forward_paged(q, b.kc, b.vc, b.plan(fa))
    fa.check()
    b.check(o, lse)


def test_explicit_scale_and_large_scores():
    b = Batch([(1, 200), (20, 300)], 4, 2, 128, 16, seed=9)
    _run(b, scale=0.3)


@pytest.mark.parametrize("lens", [[(1, 5000)], [(1, 3000), (1, 1), (1, 9000)], [(128, 4000)]])
def test_long_axis_is_split_and_joined_in_a_fixed_order(lens):
    b = Batch(lens, 4, 1, 128, 64, seed=11)
    o, lse = _run(b)
    o2, lse2 = _run(b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,window", [([(200, 5000)], 0), ([(150, 3000), (1, 40), (257, 2000)], 0),
                                         ([(300, 4000)], 1500), ([(129, 129), (64, 6000)], 0)])
def test_wide_tables(lens, window, d):
    # A table wide enough for sequences beyond L2: blocks that both tiles see are worked off in a turned order.
    b = Batch(lens, 4, 2, d, 16, seed=d + len(lens), extra_cols=40000)
    o, lse = _run(b, window=window)
    o2, lse2 = _run(b, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_many_sequences():
    r = np.random.default_rng(3)
    lens = [(int(r.integers(0, 4)), int(r.integers(0, 90))) for _ in range(1500)]
    _run(Batch(lens, 2, 1, 64, 16, seed=4))


def test_shared_prefix_pages():
    fa = fa_mod()
    b = Batch([(1, 100), (1, 100)], 4, 2, 64, 16, seed=8)
    t = b.dev["table"]
    t[1, :4] = t[0, :4]  # the first 64 tokens are one set of pages
    b.K[1][:64], b.V[1][:64] = b.K[0][:64], b.V[0][:64]
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))
    fa.check()
    b.check(o, lse)


def test_offsets_beyond_32_bits():
    # Pages whose first element lies beyond 2^32 elements of the cache.
    fa = fa_mod()
    Hkv, page, d = 8, 64, 128
    num = (1 << 32) // (Hkv * page * d) + 40
    cache = [torch.empty(num, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    b = Batch([(1, 300), (40, 200)], 16, Hkv, d, page, seed=12)
    shift = num - b.num_pages
    for c, s in zip(cache, (b.kc, b.vc)):
        c[shift:] = s
    used = b.dev["table"] >= 0
    b.dev["table"][used & (b.dev["table"] < 1 << 20)] += shift
    o, lse = fa.forward_paged(b.dev["q"], cache[0], cache[1], b.plan(fa))
    fa.check()
    b.check(o, lse)


def test_other_stream():
    fa = fa_mod()
    b = Batch([(1, 300), (30, 100)], 8, 2, 128, 16, seed=13)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    plan = b.plan(fa, stream=s)
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, stream=s)
    fa.check(stream=s)
    b.check(o, lse)
    t = torch.cuda.Stream()  # a plan used on a stream that it was not made on, and dropped at once
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, stream=t)
    del plan
    fa.check(stream=t)
    b.check(o, lse)


def test_captured_step_follows_new_lengths():
    fa = fa_mod()
    b = Batch([(1, 300), (1, 100), (1, 64)], 8, 2, 128, 16, seed=14)
    o = torch.full((b.T, b.Hq, b.d), FILL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    plan = b.plan(fa)
    fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, out=o, lse=lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        b.plan(fa, plan=plan)
        for _ in range(2):
            fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, out=o, lse=lse)
    for cut in (0, 5, 63):
        b.lens = [(1, n - cut) for n in (300, 100, 64)]
        b.dev["kv_lens"].copy_(torch.tensor([n for _, n in b.lens], dtype=torch.int32))
        o.fill_(FILL)
        lse.fill_(FILL)
        graph.replay()
        fa.check()
        for i, (ql, n) in enumerate(b.lens):
            ro, rl, to, tl = attention_ref(f64(b.q[i:i + 1]), f64(b.K[i][:n]), f64(b.V[i][:n]), n, True, 0,
                                           128 ** -0.5)
            assert_within(o[i:i + 1], ro, to, f"cut {cut} o {i}")
            assert_within(lse[i:i + 1], rl, tl, f"cut {cut} lse {i}")


def test_captured_chunks_follow_new_lengths():
    # Both kernels of a batch with chunks, captured with the plan: the cached part grows from replay to replay.
    fa = fa_mod()
    b = Batch([(40, 300), (1, 100), (200, 900)], 8, 2, 128, 16, seed=24)
    o = torch.full((b.T, b.Hq, b.d), FILL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    plan = b.plan(fa)
    fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, out=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.plan(fa, plan=plan)
        for _ in range(2):
            fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, out=o, lse=lse)
    for cut in (0, 1, 70):
        lens = [(ql, n - cut) for ql, n in b.lens]
        b.dev["kv_lens"].copy_(torch.tensor([n for _, n in lens], dtype=torch.int32))
        o.fill_(FILL)
        lse.fill_(FILL)
        graph.replay()
        fa.check()
        for i, (ql, n) in enumerate(lens):
            a = b.cu[i]
            ro, rl, to, tl = attention_ref(f64(b.q[a:a + ql]), f64(b.K[i][:n]), f64(b.V[i][:n]), n, True, 0, 128 ** -0.5,
                                           max_q=b.max_q)
            assert_within(o[a:a + ql], ro, to, f"cut {cut} o {i}")
            assert_within(lse[a:a + ql], rl, tl, f"cut {cut} lse {i}")


def test_values_beyond_a_query_do_not_reach_it_across_sequences():
    # NaN in one sequence's visible keys and values leaves the others as they are, tokens in the same tile too.
    fa = fa_mod()
    for lens in ([(1, 50), (1, 60)], [(30, 50), (30, 60)]):
        b = Batch(lens, 4, 2, 64, 16, seed=25)
        first = b.dev["table"][0, 0].item()
        b.kc[first, :, 3] = float("nan")
        b.vc[first, :, 5] = float("inf")
        o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))
        fa.check()
        a, ql, n = b.cu[1], *lens[1]
        ro, rl, to, tl = attention_ref(f64(b.q[a:]), f64(b.K[1]), f64(b.V[1]), n, True, 0, 1 / 8)
        assert_within(o[a:], ro, to, "o")
        assert_within(lse[a:], rl, tl, "lse")
        assert torch.isnan(o[0].float()).any()


def test_keys_that_a_query_does_not_see_may_be_nan():
    # A key of a later new token of the same chunk (its value is finite): masked, whatever it holds.
    fa = fa_mod()
    for new in (4, 60):
        b = Batch([(new, 100)], 4, 2, 64, 16, seed=26)
        last = b.dev["table"][0, 99 // 16].item()
        b.kc[last, :, 99 % 16] = float("nan")
        o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))
        fa.check()
        ro, rl, to, tl = attention_ref(f64(b.q), f64(b.K[0]), f64(b.V[0]), 100, True, 0, 1 / 8)
        assert_within(o[:new - 1], ro[:new - 1], to[:new - 1], "o")
        assert_within(lse[:new - 1], rl[:new - 1], tl[:new - 1], "lse")
        assert torch.isnan(o[new - 1].float()).all()


def test_agrees_with_the_dense_forward():
    # One sequence whose every token is new is fa_fwd's causal case.
    fa = fa_mod()
    N, Hq, Hkv, d = 500, 8, 2, 128
    b = Batch([(N, N)], Hq, Hkv, d, 64, seed=15)
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))
    dense = [t.transpose(0, 1)[None].contiguous().cuda() for t in (b.q, b.K[0], b.V[0])]
    od, ld = fa.forward(*dense, causal=True)
    fa.check()
    # Both are within half a bf16 step and their weights' rounding of the same value.
    assert (o.float() - od[0].transpose(0, 1).float()).abs().max() <= 2e-2
    assert (lse - ld[0].T).abs().max() <= 1e-4


# ---- what is out of range on the device is reported, and nothing out of range is touched
def _expect_index_error(fa, call):
    call()
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    fa.check()  # cleared


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("lens", [[(1, 100), (1, 40)], [(60, 100), (1, 40)]])
def test_bad_page_is_reported_and_spares_the_others(bad, lens):
    fa = fa_mod()
    b = Batch(lens, 32, 2, 64, 16, seed=16)
    b.dev["table"][0, 2] = bad
    out = []
    _expect_index_error(fa, lambda: out.extend(fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))))
    a = b.cu[1]
    ro, rl, to, tl = attention_ref(f64(b.q[a:a + 1]), f64(b.K[1]), f64(b.V[1]), 40, True, 0, 1 / 8)
    assert_within(out[0][a:a + 1], ro, to, "o")
    assert_within(out[1][a:a + 1], rl, tl, "lse")


@pytest.mark.parametrize("what,value", [("kv_lens", -1), ("kv_lens", 10 ** 6), ("cu_q", -3), ("cu_q", 10 ** 6),
                                        ("cu_q", 10 ** 3)])
def test_bad_lengths_are_reported(what, value):
    fa = fa_mod()
    b = Batch([(1, 100), (2, 40), (1, 7)], 4, 2, 64, 16, seed=17)
    b.dev[what][1] = value
    _expect_index_error(fa, lambda: fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa)))


def test_more_new_tokens_than_promised_is_reported():
    fa = fa_mod()
    b = Batch([(5, 100)], 4, 2, 64, 16, seed=18)
    b.max_q = 4
    _expect_index_error(fa, lambda: fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa)))


@pytest.mark.parametrize("field,value", [("window", 5), ("max_q", 2), ("causal", 0), ("max_pages", 8), ("T", 1)])
@pytest.mark.parametrize("lens", [[(1, 100)], [(50, 100)]])
def test_plan_of_another_batch_is_reported(field, value, lens):
    fa = fa_mod()
    b = Batch(lens, 4, 2, 64, 16, seed=19, pad=1)
    plan = b.plan(fa)
    setattr(plan._c, field, value)  # the call says something else than the plan was laid out for
    k = torch.zeros(b.T, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = f64(b.kc)
    _expect_index_error(fa, lambda: fa.forward_paged(b.dev["q"], b.kc, b.vc, plan))
    _expect_index_error(fa, lambda: fa.paged_append(None, k, k, b.kc, b.vc, plan))
    assert np.array_equal(before, f64(b.kc), equal_nan=True)


def test_plan_that_was_never_laid_out_is_reported():
    fa = fa_mod()
    b = Batch([(1, 100)], 4, 2, 64, 16, seed=20)
    plan = b.plan(fa)
    fa.check()
    plan.buffer.zero_()
    _expect_index_error(fa, lambda: fa.forward_paged(b.dev["q"], b.kc, b.vc, plan))


def test_no_sequences_and_no_tokens():
    fa = fa_mod()
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = fa.paged_plan(z, z[:0], torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 4, 1, 16, 4, 2, 64)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    fa.forward_paged(q, kc, kc, plan)
    plan = fa.paged_plan(torch.cat([z, z]), z, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), 0, 0, 16, 4, 2, 64)
    o, lse = fa.forward_paged(q[:0], kc, kc, plan)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    fa.check()
