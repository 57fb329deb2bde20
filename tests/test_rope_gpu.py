"""Rotary positions (fa_rope, fa_rope_bwd) and the rotating append to a paged cache (fa_paged_append) against fp64."""

import math

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch, assert_within, attention_ref, f64, rope_ref, rotary

pytestmark = pytest.mark.gpu


def _rotary(fa, rot, theta=1.0e4, interleaved=False, axes=None):
    return fa.Rotary(rotary(rot, theta).cuda(), interleaved=interleaved, axes=axes)


def _pair_positions(pos, rot, axes):
    """[.., N] per axis -> [.., N, rot / 2]."""
    pos = np.asarray(pos, dtype=np.float64)
    if axes is None:
        return np.repeat(pos[..., None], rot // 2, -1)
    return np.stack([pos[a] for a in axes], -1)


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("N", [1, 2, 3, 5, 17, 130])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64), (64, 16), (128, 96), (128, 112), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_and_backward(N, d, rot, interleaved):
    fa = fa_mod()
    B, Hq, Hkv = 2, 3, 1
    q, k = _randn(B, Hq, N, d, seed=N), _randn(B, Hkv, N, d, seed=N + 1)
    pos = torch.arange(N, dtype=torch.int32) * 37 + 5
    r = _rotary(fa, rot, interleaved=interleaved)
    pp = _pair_positions(pos.numpy(), rot, None)
    for fn, inv in ((fa.rope, False), (fa.rope_backward, True)):
        got = fn(q.cuda(), k.cuda(), pos.cuda(), r)
        fa.check()
        for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
            ref, tol = rope_ref(f64(x), pp, rotary(rot), interleaved, inv)
            assert y.is_contiguous()
            assert_within(y, ref, tol, f"{fn.__name__} {name}")


def test_gradient_against_differences():
    # <g, R(x + h e) - R(x - h e)> / 2h with the fp64 rotation, for the gradient that the kernel returns.
    fa = fa_mod()
    N, d = 3, 64
    x, g = _randn(1, 1, N, d, seed=1), _randn(1, 1, N, d, seed=2)
    pos = torch.tensor([3, 1000, 70000], dtype=torch.int32)
    pp = _pair_positions(pos.numpy(), d, None)
    grad, _ = fa.rope_backward(g.cuda(), None, pos.cuda(), _rotary(fa, d))
    fa.check()
    num = np.zeros((1, 1, N, d))
    h = 1e-3
    for i in np.ndindex(num.shape):
        e = np.zeros(num.shape)
        e[i] = h
        up, down = (rope_ref(f64(x) + s * e, pp, rotary(d))[0] for s in (1, -1))
        num[i] = (f64(g) * (up - down)).sum() / (2 * h)
    _, tol = rope_ref(f64(g), pp, rotary(d), inverse=True)
    assert_within(grad, num, tol + 1e-9, "gradient")  # 1e-9: the differences' own rounding, 2^-52 / h


@pytest.mark.parametrize("start", [0, 131072, 2 ** 24 + 1, 2 ** 31 - 64, -2 ** 31])
@pytest.mark.parametrize("theta", [1.0e4, 5.0e5])
def test_far_positions_keep_their_angles(start, theta):
    fa = fa_mod()
    N, d = 64, 128
    q = _randn(1, 2, N, d, seed=3)
    pos = (torch.arange(N, dtype=torch.int64) + start).to(torch.int32)
    got, _ = fa.rope(q.cuda(), None, pos.cuda(), _rotary(fa, d, theta))
    fa.check()
    ref, tol = rope_ref(f64(q), _pair_positions(pos.numpy(), d, None), rotary(d, theta))
    # Per position the angle carries 2^-53 of the double that the frequency's turns are kept in (2^-53 as well in the
    # reference's own product): 2 * 2^-53 * 2^31 rad at the ends.
    ends = 2.0 ** -52 * abs(float(start) + N) * (np.abs(f64(q)).max() * 2)
    assert_within(got, ref, tol + ends, f"start {start}")


@pytest.mark.parametrize("d,sections", [(64, (8, 12, 12)), (128, (16, 24, 24)), (128, (1, 62, 1)), (64, (5, 6, 7, 14))])
@pytest.mark.parametrize("per_batch", [False, True])
def test_several_axes(d, sections, per_batch):
    fa = fa_mod()
    B, N = 2, 45
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    shape = (len(sections), B, N) if per_batch else (len(sections), N)
    pos = torch.randint(0, 5000, shape, generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    q, k = _randn(B, 4, N, d, seed=5), _randn(B, 2, N, d, seed=6)
    got = fa.rope(q.cuda(), k.cuda(), pos.cuda(), _rotary(fa, d, axes=axes))
    fa.check()
    pp = _pair_positions(pos.numpy(), d, axes)
    pp = pp[:, None] if per_batch else pp
    for x, y in ((q, got[0]), (k, got[1])):
        ref, tol = rope_ref(f64(x), np.broadcast_to(pp, x.shape[:-1] + (d // 2,)), rotary(d))
        assert_within(y, ref, tol)


def test_interleaved_axes_any_assignment():
    fa = fa_mod()
    axes = [i % 3 for i in range(32)]
    pos = torch.randint(0, 999, (3, 20), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    q = _randn(1, 2, 20, 64, seed=8)
    got, _ = fa.rope(q.cuda(), None, pos.cuda(), _rotary(fa, 64, interleaved=True, axes=axes))
    fa.check()
    ref, tol = rope_ref(f64(q), _pair_positions(pos.numpy(), 64, axes), rotary(64), True)
    assert_within(got, ref, tol)


def test_views_in_place_and_other_stream():
    fa = fa_mod()
    B, N, Hq, Hkv, d = 2, 33, 4, 2, 128
    base = _randn(B, N, Hq + 2 * Hkv, d, seed=9)
    pos = torch.randint(0, 9999, (B, N), generator=torch.Generator().manual_seed(10), dtype=torch.int32)
    r = _rotary(fa, d)
    pp = _pair_positions(pos.numpy(), d, None)[:, None]
    fused = base.cuda()
    q, k = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hkv].transpose(1, 2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = fa.rope(q, k, pos.cuda(), r, stream=s)
    fa.check(stream=s)
    refs = [rope_ref(f64(base[:, :, a:b].transpose(1, 2)), pp, rotary(d)) for a, b in ((0, Hq), (Hq, Hq + Hkv))]
    for y, (ref, tol) in zip(out, refs):
        assert_within(y, ref, tol)
    fa.rope(q, k, pos.cuda(), r, q_out=q, k_out=k)  # in place, in the fused tensor
    fa.check()
    for y, (ref, tol) in zip((q, k), refs):
        assert_within(y, ref, tol)
    assert torch.equal(fused[:, :, Hq + Hkv:].cpu(), base[:, :, Hq + Hkv:])  # the values are as they were


def test_captured_backward_while_an_eager_graph_lives():
    # The calls hold no autograd state of their own: capturing one next to a live eager graph is safe.
    fa = fa_mod()
    x = torch.randn(2, 2, 8, 64, device="cuda", requires_grad=True)
    y = (x * 2).sum()
    g = x.detach().to(torch.bfloat16)
    pos, r = torch.arange(8, dtype=torch.int32, device="cuda"), _rotary(fa, 64)
    want = fa.rope_backward(g, None, pos, r)[0]
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.rope_backward(g, None, pos, r, q_out=out)
    graph.replay()
    fa.check()
    assert torch.equal(out, want)
    y.backward()


# ---------------------------------------------------------------------------------------------- append
def _append_case(lens, Hq, Hkv, d, page, rot, interleaved=False, axes=None, layout="phsd", pad=0, lead=0, seed=0,
                 with_q=True):
    fa = fa_mod()
    b = Batch(lens, Hq, Hkv, d, page, seed=seed, layout=layout, pad=pad, lead=lead)
    T = b.T
    k, v = _randn(T, Hkv, d, seed=seed + 1), _randn(T, Hkv, d, seed=seed + 2)
    r = _rotary(fa, rot, 5.0e5, interleaved, axes) if rot else None
    positions = None
    if axes is not None:
        positions = torch.randint(0, 3000, (max(axes) + 1, T), generator=torch.Generator().manual_seed(seed),
                                  dtype=torch.int32)
    before = f64(b.kc), f64(b.vc)
    q_out = torch.full((T, Hq, d), -7.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    fa.paged_append(b.q.cuda() if with_q else None, k.cuda(), v.cuda(), b.kc, b.vc, b.plan(fa), r,
                    positions.cuda() if positions is not None else None, q_out=q_out)
    fa.check()
    kc, vc = before
    tol_k = np.zeros_like(kc)
    want_q, tol_q = np.full((T, Hq, d), -7.0), np.zeros((T, Hq, d))
    for i, (ql, n) in enumerate(lens):
        for j in range(ql):
            t, pos = b.cu[i] + j, n - ql + j
            if rot:
                p = np.full(rot // 2, float(pos)) if axes is None else np.array([float(positions[a, t]) for a in axes])
                want_q[t], tol_q[t] = rope_ref(f64(b.q[t]), p, rotary(rot, 5.0e5), interleaved)
                kk, tk = rope_ref(f64(k[t]), p, rotary(rot, 5.0e5), interleaved)
            else:
                kk, tk = f64(k[t]), 0.0
            page_id = int(b.table[i, pos // page])
            kc[page_id, :, pos % page], tol_k[page_id, :, pos % page] = kk, tk
            vc[page_id, :, pos % page] = f64(v[t])
    assert_within(b.kc, kc, tol_k, "k cache")  # every other slot as it was, NaN among them
    assert_within(b.vc, vc, 0.0, "v cache")
    if with_q:
        assert_within(q_out, want_q, tol_q, "q")


@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 100), (1, 16), (1, 17)], [(5, 5), (0, 9), (33, 70), (1, 64)],
                                  [(0, 0), (0, 4), (2, 2), (0, 0)], [(1, 7)] * 37])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 64, True), (128, 64, False), (64, 0, False)])
@pytest.mark.parametrize("page", [16, 128])
def test_append(lens, d, rot, interleaved, page):
    _append_case(lens, 4, 2, d, page, rot, interleaved, pad=3, lead=2, seed=len(lens), with_q=rot > 0)


@pytest.mark.parametrize("layout", ["pshd", "both"])
def test_append_layouts_and_axes(layout):
    _append_case([(3, 40), (20, 20)], 6, 3, 64, 32, 64, axes=[0] * 8 + [1] * 12 + [2] * 12, layout=layout, seed=21)


def test_append_without_queries_and_odd_heads():
    _append_case([(3, 40), (20, 21)], 7, 7, 128, 64, 128, seed=22, with_q=False)


def _index_error(fa, call):
    call()
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    fa.check()


@pytest.mark.parametrize("bad", ["page", "short"])
def test_append_out_of_range_is_reported_and_writes_nothing_there(bad):
    fa = fa_mod()
    b = Batch([(2, 40), (1, 20)], 4, 2, 64, 16, seed=23)
    if bad == "page":
        b.dev["table"][0, 2] = b.num_pages  # positions 38, 39
    else:
        b.dev["kv_lens"][0] = 1  # two new tokens, one token in all
    before = f64(b.kc)
    k = _randn(3, 2, 64, seed=24).cuda()
    _index_error(fa, lambda: fa.paged_append(None, k, k, b.kc, b.vc, b.plan(fa)))
    after = f64(b.kc)
    same = (before == after) | (np.isnan(before) & np.isnan(after))
    changed = {(int(p), int(s)) for p, _, s, _ in np.argwhere(~same)}
    ok = {(int(b.table[1, 1]), 3)} | ({(int(b.table[0, 0]), 0)} if bad == "short" else set())
    assert changed <= ok and (int(b.table[1, 1]), 3) in changed


def test_decode_loop_follows_the_dense_forward():
    # A prompt in two chunks, then token by token: rotated, appended and attended, against the whole sequence rotated
    # and attended at once. Each result is within its own rounding of the fp64 value.
    fa = fa_mod()
    N, Hq, Hkv, d, page = 150, 4, 2, 64, 16
    qkv = _randn(N, Hq + 2 * Hkv, d, seed=31).cuda()
    r = _rotary(fa, d)
    P = (N + page - 1) // page
    kc = torch.full((P, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("inf"))
    table = torch.randperm(P, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None].cuda()
    outs, lses = [], []
    steps = [(0, 90), (90, 130)] + [(i, i + 1) for i in range(130, N)]
    for a, e in steps:
        x = qkv[a:e]
        cu = torch.tensor([0, e - a], dtype=torch.int32, device="cuda")
        plan = fa.paged_plan(cu, torch.tensor([e], dtype=torch.int32, device="cuda"), table, e - a, e - a, page, Hq, Hkv,
                             d)
        q = fa.paged_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, plan, r)
        o, lse = fa.forward_paged(q, kc, vc, plan)
        outs.append(o)
        lses.append(lse)
    fa.check()
    o, lse = torch.cat(outs), torch.cat(lses)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    h = qkv.transpose(0, 1)[None]
    qd, kd = fa.rope(h[:, :Hq], h[:, Hq:Hq + Hkv], pos, r)
    fa.check()
    # The rotated tensors are the same bits; the attention over them is checked against fp64.
    ro, rl, to, tl = attention_ref(f64(qd[0].transpose(0, 1)), f64(kd[0].transpose(0, 1)),
                                   f64(qkv[:, Hq + Hkv:]), N, True, 0, 1 / math.sqrt(d))
    assert_within(lse, rl, tl, "lse")
    assert_within(o, ro, to, "o")
    od, ld = fa.forward(qd, kd, h[:, Hq + Hkv:].contiguous(), causal=True)
    fa.check()
    assert (lse - ld[0].T).abs().max() <= 1e-4


def test_training_step_gradients():
    # rope -> fa.forward / fa.backward -> rope_backward against fp64 differences of the whole step.
    import oracle

    fa = fa_mod()
    B, Hq, Hkv, N, d = 1, 2, 1, 40, 64
    q, k, v, do = (_randn(B, h, N, d, seed=40 + i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    pos, r = torch.arange(N, dtype=torch.int32).cuda(), _rotary(fa, d)
    pp = _pair_positions(np.arange(N), d, None)
    qr, kr = fa.rope(q.cuda(), k.cuda(), pos, r)
    o, lse = fa.forward(qr, kr, v.cuda(), True)
    dqr, dkr, _ = fa.backward(qr, kr, v.cuda(), o, do.cuda(), lse, True)
    dq, dk = fa.rope_backward(dqr, dkr, pos, r)
    fa.check()
    scale = 1 / math.sqrt(d)

    def loss(qx, kx):
        a = rope_ref(qx, pp, rotary(d))[0]
        c = rope_ref(kx, pp, rotary(d))[0]
        return (oracle.attention_forward(a, c, f64(v), True, scale)[0] * f64(do)).sum()

    rng = np.random.default_rng(0)
    for name, grad in (("q", dq), ("k", dk)):
        for _ in range(3):  # directional derivatives; the attention backward's bound of 2e-2 of the norms
            e = rng.standard_normal(grad.shape)
            h = 1e-5
            args = [(f64(q) + s * h * e, f64(k)) if name == "q" else (f64(q), f64(k) + s * h * e) for s in (1, -1)]
            num = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            g = f64(grad)
            assert abs((g * e).sum() - num) <= 2e-2 * np.linalg.norm(g) * np.linalg.norm(e) / math.sqrt(g.size) * 3
