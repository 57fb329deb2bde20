"""The 4-bit cache, weights and eviction captured into graphs, on other streams, with foreign plans, and between guard bytes."""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4
from paged_util import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def step(fa, b, plan, cache, w, kv, keep, to, outs):
    """A serving step as a layer runs it, into given outputs."""
    fa.paged_append4(None, kv[:, :b.Hkv], kv[:, b.Hkv:], cache, plan)
    fa.forward_paged4(b.dev["q"], cache, plan, out=outs[0], lse=outs[1])
    fa.paged_weights(b.dev["q"], outs[1], cache, w, plan)
    fa.paged_evict(w, cache, plan, keep, to, max_keep=40, sinks=2, recent=4, kept=outs[2], kv_lens=outs[3])


@pytest.mark.parametrize("d,ql", [(128, 1), (64, 3), (128, 40)])
def test_captured_step_follows_new_lengths(fa, d, ql):
    lens = [(ql, 200), (ql, 97), (ql, 64)]
    b = Batch4(fa, lens, 4, 2, d, 16, seed=ql)
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(b.T, 4, d, generator=g).to(torch.bfloat16).cuda()
    extra = 9
    pages = b.num_pages + extra
    to = (torch.arange(9, dtype=torch.int32) + b.num_pages).view(3, 3).cuda()
    keep = torch.full((3,), 40, dtype=torch.int32, device="cuda")

    def state():
        cache = fa.PagedCache4.empty(pages, 2, 16, d)
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)):
            x.zero_()
            x[:b.num_pages] = y
        w = torch.rand(pages, 2, 16, generator=torch.Generator().manual_seed(2)).cuda()
        outs = (torch.zeros(b.T, 4, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(b.T, 4, device="cuda"),
                torch.zeros(3, 2, 40, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"))
        return cache, w, outs

    cache, w, outs = state()
    plan = b.plan(fa)
    step(fa, b, plan, cache, w, kv, keep, to, outs)
    fa.check()
    cache, w, outs = state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.plan(fa, plan=plan)
        step(fa, b, plan, cache, w, kv, keep, to, outs)
    for lengths in ([200, 97, 64], [150, 60, 41], [43, 97, 40]):
        fresh_cache, fresh_w, fresh_outs = state()
        b.dev["kv_lens"].copy_(torch.tensor(lengths, dtype=torch.int32))
        step(fa, b, b.plan(fa), fresh_cache, fresh_w, kv, keep, to, fresh_outs)
        c2, w2, _ = state()
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, w), (c2.k, c2.v, c2.k_scale, c2.v_scale, w2)):
            x.copy_(y)
        graph.replay()
        fa.check()
        for x, y in zip((*outs, w, cache.k, cache.v_scale), (*fresh_outs, fresh_w, fresh_cache.k, fresh_cache.v_scale)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_streams_at_once_with_a_plan_each(fa):
    bs = [Batch4(fa, [(1, 3000), (1, 17), (30, 900)], 8, 2, 128, 16, seed=i) for i in (1, 2)]
    streams = [torch.cuda.Stream() for _ in bs]
    want = []
    for b in bs:
        want.append(fa.forward_paged4(b.dev["q"], b.cache, b.plan(fa)))
    fa.check()
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for b, s in zip(bs, streams):
            s.wait_stream(torch.cuda.current_stream())
            plan = b.plan(fa, stream=s)
            got.append(fa.forward_paged4(b.dev["q"], b.cache, plan, stream=s))
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_a_plan_of_other_sizes_is_reported(fa):
    b = Batch4(fa, [(1, 100), (1, 40)], 4, 2, 64, 16, seed=1)
    plan = b.plan(fa)
    plan.buffer.zero_()  # no plan at all
    w = torch.zeros(b.num_pages, 2, 16, device="cuda")
    lse = torch.zeros(2, 4, device="cuda")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    to = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for call in (lambda: fa.forward_paged4(b.dev["q"], b.cache, plan), lambda: fa.paged_append4(None, x, x, b.cache, plan),
                 lambda: fa.paged_weights(b.dev["q"], lse, b.cache, w, plan),
                 lambda: fa.paged_evict(w, b.cache, plan, to[:, 0].contiguous(), to, max_keep=8)):
        call()
        with pytest.raises(fa.FAError) as e:
            fa.check()
        assert e.value.status == -8


def guarded(shape, dtype, fill=0x5A):
    """A tensor of ``shape`` between 4 KB of guard bytes on either side, and the check of those."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 8192,), fill, dtype=torch.uint8, device="cuda")
    t = raw[4096:4096 + n].view(dtype).view(shape)

    def intact():
        return bool((raw[:4096] == fill).all()) and bool((raw[4096 + n:] == fill).all())

    return t, intact


@pytest.mark.parametrize("d,heads", [(64, (6, 3)), (128, (5, 1))])
def test_nothing_is_written_beyond_the_buffers(fa, d, heads):
    Hq, Hkv = heads
    b = Batch4(fa, [(1, 77), (9, 9), (0, 5), (50, 333), (2, 16)], Hq, Hkv, d, 16, seed=4, pad=1)
    guards = []

    def make(shape, dtype):
        t, ok = guarded(shape, dtype)
        guards.append(ok)
        return t

    page = (b.num_pages + 12, Hkv, 16)
    parts = [make(page + (d // 2,), torch.uint8), make(page + (d // 2,), torch.uint8), make(page + (d // 32,), torch.bfloat16),
             make(page + (d // 32,), torch.bfloat16)]
    for x, y in zip(parts, (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)):
        x.zero_()
        x[:b.num_pages] = y
    cache = fa.PagedCache4(*parts)
    w = make(page, torch.float32)
    w.fill_(0.5)
    out_w = make(page, torch.float32)
    o, lse = make((b.T, Hq, d), torch.bfloat16), make((b.T, Hq), torch.float32)
    ko, vo = make((b.T, Hkv, d), torch.bfloat16), make((b.T, Hkv, d), torch.bfloat16)
    kept, lens = make((5, Hkv, 33), torch.int32), make((5,), torch.int32)
    plan = b.plan(fa)
    n = plan.ws_bytes
    plan.workspace, ok = guarded((n,), torch.uint8)
    guards.append(ok)
    x = torch.randn(b.T, 2 * Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    fa.paged_append4(None, x[:, :Hkv], x[:, Hkv:], cache, plan, k_out=ko, v_out=vo)
    fa.forward_paged4(b.dev["q"], cache, plan, out=o, lse=lse)
    fa.paged_weights(b.dev["q"], lse, cache, w, plan, out=out_w)
    to = torch.zeros(5, 3, dtype=torch.int32)
    to.view(-1)[:12] = torch.arange(12, dtype=torch.int32) + b.num_pages
    keep = torch.tensor([33, 33, 33, 33, 0], dtype=torch.int32).cuda()
    fa.paged_evict(w, cache, plan, keep, to.cuda(), max_keep=33, kept=kept, kv_lens=lens)
    fa.check()
    assert all(g() for g in guards)
    assert lens.tolist() == [33, 9, 5, 33, 0]
    assert np.isfinite(f64(o)[:62]).all()


def test_the_smallest_and_the_empty(fa):
    for lens in ([(1, 1)], [(0, 0)], []):
        b = Batch4(fa, lens, 1, 1, 64, 16, seed=1)
        plan = b.plan(fa)
        x = torch.ones(b.T, 2, 64, dtype=torch.bfloat16, device="cuda")
        fa.paged_append4(None, x[:, :1], x[:, 1:], b.cache, plan)
        o, lse = fa.forward_paged4(b.dev["q"], b.cache, plan)
        w = torch.zeros(b.num_pages, 1, 16, device="cuda")
        fa.paged_weights(b.dev["q"], lse, b.cache, w, plan)
        kept, n = fa.paged_evict(w, b.cache, plan, torch.ones(len(lens), dtype=torch.int32, device="cuda"),
                                 torch.full((len(lens), 1), b.num_pages - 1, dtype=torch.int32, device="cuda"), max_keep=1)
        fa.check()
        if lens == [(1, 1)]:
            page = int(b.table[0, 0])
            # The one key has all the weight, and ones are stored exactly (s = 0.140625, u = 15: 0.984375).
            assert abs(float(w[page, 0, 0]) - 1) < 2.0 ** -18 and bool((o == 0.984375).all())
            assert kept.tolist() == [[[0]]] and n.tolist() == [1]
