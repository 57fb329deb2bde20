"""Eviction by weight: places, lengths and every byte moved, exactly."""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def choose(w, n, keep, sinks, recent):
    """The places that stay of n tokens with weights w."""
    new = min(n, keep)
    a = min(sinks, new)
    b = n - min(recent, new - a)
    m = new - a - (n - b)
    mid = np.where(np.isnan(w[a:b]), np.inf, w[a:b]).astype(np.float64)
    nan = np.isnan(w[a:b])
    order = sorted(range(b - a), key=lambda i: (not nan[i], -mid[i], i))[:m]
    return list(range(a)) + sorted(a + i for i in order) + list(range(b, n))


class Setup:
    def __init__(self, fa, lens, Hkv, d, page, keep, max_keep=None, seed=0, kind="random", table_pad=1):
        g = torch.Generator().manual_seed(seed)
        self.fa, self.lens, self.Hkv, self.d, self.page = fa, lens, Hkv, d, page
        self.keep = keep if isinstance(keep, list) else [keep] * len(lens)
        self.max_keep = max(self.keep + [0]) if max_keep is None else max_keep
        S = len(lens)
        have = [(n + page - 1) // page for n in lens]
        want = [(min(n, k) + page - 1) // page for n, k in zip(lens, self.keep)]
        self.pages = sum(have) + sum(want) + 2
        order = torch.randperm(self.pages, generator=g).tolist()
        cols = max(have + [1]) + 1
        out_cols = max((self.max_keep + page - 1) // page, 1) + table_pad
        self.table = torch.full((S, cols), -5, dtype=torch.int32)
        self.to = torch.full((S, out_cols), 1 << 29, dtype=torch.int32)
        for i in range(S):
            self.table[i, :have[i]] = torch.tensor([order.pop() for _ in range(have[i])], dtype=torch.int32)
            self.to[i, :want[i]] = torch.tensor([order.pop() for _ in range(want[i])], dtype=torch.int32)
        shape = (self.pages, Hkv, page)
        if kind == "random":
            self.w = torch.exp(3 * torch.randn(shape, generator=g))
        elif kind == "ties":
            self.w = torch.randint(0, 4, shape, generator=g).float()
        elif kind == "equal":
            self.w = torch.full(shape, 0.25)
        else:  # of all kinds
            self.w = torch.randn(shape, generator=g)
            pick = torch.randint(0, 8, shape, generator=g)
            for i, v in enumerate((float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 1e-42)):
                self.w[pick == i] = v
        self.tensors = [torch.randint(0, 256, shape + (n,), generator=g, dtype=torch.int64).to(torch.uint8)
                        for n in (2 * d, 2 * d, d // 2, 1, 6)]
        self.plan = fa.paged_plan(torch.arange(S + 1, dtype=torch.int32).cuda() * 0, torch.tensor(lens, dtype=torch.int32).cuda(),
                                  self.table.cuda(), num_tokens=0, max_q=0, page_size=page, Hq=Hkv, Hkv=Hkv, d=d)

    def run(self, sinks, recent, check=True):
        fa = self.fa
        w, t = self.w.cuda(), [x.cuda() for x in self.tensors]
        kept, lens = fa.paged_evict(w, t, self.plan, torch.tensor(self.keep, dtype=torch.int32).cuda(), self.to.cuda(),
                                    max_keep=self.max_keep, sinks=sinks, recent=recent)
        if check:
            fa.check()
        want_kept = np.full((len(self.lens), self.Hkv, self.max_keep), -1)
        want = [x.clone() for x in self.tensors + [self.w]]
        for i, (n, keep) in enumerate(zip(self.lens, self.keep)):
            for h in range(self.Hkv):
                at = np.arange(n)
                wi = self.w[self.table[i, at // self.page].long(), h, at % self.page].numpy() if n else np.zeros(0)
                places = choose(wi, n, keep, sinks, recent)
                want_kept[i, h, :len(places)] = places
                for x, src in zip(want, self.tensors + [self.w]):
                    for a, p in enumerate(places):
                        x[self.to[i, a // self.page], h, a % self.page] = src[self.table[i, p // self.page], h, p % self.page]
        np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
        assert lens.tolist() == [min(n, k) for n, k in zip(self.lens, self.keep)]
        for x, y in zip(want, t + [w]):
            assert torch.equal(x.view(torch.uint8), y.cpu().contiguous().view(torch.uint8))


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "all kinds"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 16), (1, 0), (0, 33), (200, 5), (3, 300)])
def test_what_stays(fa, kind, sinks, recent):
    Setup(fa, [300, 1, 0, 100, 101, 64, 513], 2, 64, 16, 100, seed=sinks, kind=kind).run(sinks, recent)


@pytest.mark.parametrize("d,page,Hkv", [(64, 16, 1), (128, 64, 5), (128, 256, 2)])
@pytest.mark.parametrize("keep", [0, 1, 31, 32, 33, 2000])
def test_sizes(fa, d, page, Hkv, keep):
    Setup(fa, [700, 33, 5], Hkv, d, page, keep, max_keep=max(keep, 1) if keep < 2000 else 2000, seed=keep).run(4, 8)


def test_a_bound_of_its_own_for_each_sequence(fa):
    Setup(fa, [100, 200, 300, 50], 3, 64, 32, [10, 200, 0, 64], max_keep=250, seed=1).run(2, 3)


@pytest.mark.parametrize("kind", ["random", "ties"])
def test_more_weights_than_shared_memory_holds(fa, kind):
    s = Setup(fa, [50000], 1, 64, 256, 777, seed=2, kind=kind)
    s.tensors = s.tensors[3:]
    s.run(4, 64)


@pytest.mark.parametrize("kind", ["random", "ties", "all kinds"])
def test_more_weights_than_shared_memory_holds_and_many_sequences(fa, kind):
    """A CTA per sequence and head, which reads the weights again in each pass."""
    s = Setup(fa, [50000, 45057, 45056, 0, 3] + [20] * 75, 2, 64, 256, 333, seed=4, kind=kind)
    s.tensors = s.tensors[3:]
    s.run(4, 64)


@pytest.mark.parametrize("kind", ["ties", "all kinds"])
def test_more_weights_than_a_cluster_holds(fa, kind):
    s = Setup(fa, [370000], 1, 64, 256, 777, seed=5, kind=kind)
    s.tensors = s.tensors[3:]
    s.run(4, 64)


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "all kinds"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 33), (1000, 5), (3, 1000)])
@pytest.mark.parametrize("lens", [[2100, 40, 0, 2047], [17000, 5000, 300], [9000]])  # clusters of 2 to 8
def test_what_stays_by_clusters(fa, kind, sinks, recent, lens):
    s = Setup(fa, lens, 2, 64, 64, 300, seed=sinks + len(lens), kind=kind)
    s.tensors = s.tensors[3:]
    s.run(sinks, recent)


def test_lengths_and_pages_out_of_range(fa):
    s = Setup(fa, [100, 200, 90], 2, 64, 16, [50, 60, 40], seed=3)
    s.keep[1] = 61  # above max_keep: nothing of it stays
    s.to[2, 1] = s.pages  # its slots 16 .. 31 have no page
    w, t = s.w.cuda(), [x.cuda() for x in s.tensors]
    kept, lens = fa.paged_evict(w, t, s.plan, torch.tensor(s.keep, dtype=torch.int32).cuda(), s.to.cuda(), max_keep=60, sinks=0,
                                recent=0)
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    assert lens.tolist() == [50, 0, 40] and bool((kept[1] == -1).all())
    for x, y in zip(s.tensors + [s.w], t + [w]):
        y = y.cpu()
        untouched = torch.ones(s.pages, dtype=torch.bool)
        untouched[s.to[0, :4].long()] = False
        untouched[s.to[2, [0, 2]].long()] = False
        assert torch.equal(x[untouched].view(torch.uint8), y[untouched].view(torch.uint8))
        for a in (0, 15, 32, 39):  # of the third sequence: where its pages exist
            p = int(kept[2, 1, a])
            assert torch.equal(x[s.table[2, p // 16], 1, p % 16], y[s.to[2, a // 16], 1, a % 16])


def test_smaller_caches_as_they_are_used(fa):
    """Tokens into a 4-bit cache, attention, their weights, eviction, and a step over what is left."""
    d, Hq, Hkv, page = 128, 8, 2, 16
    b = Batch4(fa, [(3, 200), (1, 90), (2, 40)], Hq, Hkv, d, page, seed=5)
    g = torch.Generator().manual_seed(2)
    new = torch.randn(b.T, 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    extra = 12
    cache = fa.PagedCache4.empty(b.num_pages + extra, Hkv, page, d)
    for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)):
        x.zero_()
        x[:b.num_pages] = y
    weights = torch.zeros(b.num_pages + extra, Hkv, page, device="cuda")
    plan = b.plan(fa)
    seen = [torch.empty(b.T, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.paged_append4(None, new[:, :Hkv], new[:, Hkv:], cache, plan, k_out=seen[0], v_out=seen[1])
    for i, (ql, n) in enumerate(b.lens):
        b.K[i][n - ql:] = seen[0][b.cu[i]:b.cu[i] + ql].cpu()
        b.V[i][n - ql:] = seen[1][b.cu[i]:b.cu[i] + ql].cpu()
    o, lse = fa.forward_paged4(b.dev["q"], cache, plan)
    fa.paged_weights(b.dev["q"], lse, cache, weights, plan)
    fa.check()
    b.check(o, lse)
    keep = torch.full((3,), 48, dtype=torch.int32, device="cuda")
    to = (torch.arange(12, dtype=torch.int32) + b.num_pages).view(3, 4).cuda()
    w = weights.cpu()
    kept, lens = fa.paged_evict(weights, cache, plan, keep, to, max_keep=48, sinks=2, recent=8)
    fa.check()
    assert lens.tolist() == [48, 48, 40]
    for i, (_, n) in enumerate(b.lens):
        at = np.arange(n)
        for h in range(Hkv):
            want = choose(w[b.table[i, at // page].long(), h, at % page].numpy(), n, 48, 2, 8)
            assert kept[i, h, :len(want)].tolist() == want
    # The next step: one token each, at the end of the shorter caches.
    step = Batch4(fa, [(1, int(n) + 1) for n in lens], Hq, Hkv, d, page, seed=6)
    plan2 = fa.paged_plan(step.dev["cu_q"], step.dev["kv_lens"], to, num_tokens=3, max_q=1, page_size=page, Hq=Hq, Hkv=Hkv, d=d)
    x = torch.randn(3, 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    ko, vo = (torch.empty(3, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.paged_append4(None, x[:, :Hkv], x[:, Hkv:], cache, plan2, k_out=ko, v_out=vo)
    o, lse = fa.forward_paged4(step.dev["q"], cache, plan2)
    fa.check()
    for i, n in enumerate(lens.tolist()):
        K, V = torch.empty(n + 1, Hkv, d), torch.empty(n + 1, Hkv, d)
        for h in range(Hkv):
            p = kept[i, h, :n].long().cpu()
            K[:n, h], V[:n, h] = b.K[i][p, h].float(), b.V[i][p, h].float()
        K[n], V[n] = ko[i].cpu().float(), vo[i].cpu().float()
        step.K[i], step.V[i] = K.to(torch.bfloat16), V.to(torch.bfloat16)
    step.check(o, lse)
