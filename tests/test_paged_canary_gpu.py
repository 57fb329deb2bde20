"""Guard bytes around every buffer that the rotary, append and paged-attention entry points write: plan, workspace,
outputs, caches."""

import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch
from test_canary_gpu import Guarded

pytestmark = pytest.mark.gpu


def _guarded_plan(fa, b, window):
    plan = b.plan(fa, True, window)
    g, w = Guarded(plan.buffer.shape, torch.uint8), Guarded(plan.workspace.shape, torch.uint8)
    plan.buffer, plan.workspace, plan._c.plan = g.t, w.t, g.t.data_ptr()
    return b.plan(fa, True, window, plan=plan), g, w


def _guarded_like(t):
    g = Guarded(t.shape, t.dtype)
    g.t.copy_(t)
    return g


@pytest.mark.parametrize("lens", [[(1, 5000)], [(1, n) for n in range(0, 900, 13)], [(4, 700)] * 5, [(4, 90)] * 60,
                                  [(150, 900), (1, 700), (0, 3), (3, 2)], [(700, 2000)], [(1, 1)] * 1100, [(0, 0)]])
@pytest.mark.parametrize("heads", [(8, 1), (6, 3), (130, 1)])
@pytest.mark.parametrize("d,window", [(64, 0), (128, 333)])
def test_attention_stays_inside_its_buffers(lens, heads, d, window):
    fa = fa_mod()
    b = Batch(lens, *heads, d, 16, seed=len(lens), pad=1)
    plan, g, w = _guarded_plan(fa, b, window)
    k, v = _guarded_like(b.kc), _guarded_like(b.vc)
    o, lse = Guarded(b.q.shape, torch.bfloat16), Guarded((b.T, b.Hq), torch.float32)
    fa.forward_paged(b.dev["q"], k.t, v.t, plan, out=o.t, lse=lse.t)
    fa.check()
    for name, x in (("plan", g), ("workspace", w), ("o", o), ("lse", lse), ("k", k), ("v", v)):
        assert x.intact(), name


@pytest.mark.parametrize("lens", [[(1, 33)], [(1, n) for n in range(1, 90)], [(70, 128), (0, 4), (1, 17), (5, 5)]])
@pytest.mark.parametrize("heads", [(8, 1), (6, 3)])
@pytest.mark.parametrize("d,width", [(64, 32), (128, 64), (64, 8)])
def test_append_stays_inside_its_buffers(lens, heads, d, width):
    fa = fa_mod()
    b = Batch(lens, *heads, d, 16, seed=len(lens), pad=1)
    plan, g, w = _guarded_plan(fa, b, 0)
    k, v, qo = _guarded_like(b.kc), _guarded_like(b.vc), Guarded(b.q.shape, torch.bfloat16)
    rot = fa.Rotary(torch.rand(width, device="cuda"), interleaved=width == 8)
    new = torch.randn(b.T, b.Hkv, d, device="cuda").to(torch.bfloat16)
    fa.paged_append(b.dev["q"], new, new, k.t, v.t, plan, rot, q_out=qo.t)
    fa.check()
    for name, x in (("plan", g), ("workspace", w), ("q", qo), ("k", k), ("v", v)):
        assert x.intact(), name


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 3, 1, 129), (1, 8, 2, 1000)])
@pytest.mark.parametrize("d,width", [(64, 32), (128, 64), (128, 24)])
def test_rope_stays_inside_its_buffers(shape, d, width):
    fa = fa_mod()
    B, Hq, Hkv, N = shape
    q = torch.randn(B, Hq, N, d, device="cuda").to(torch.bfloat16)
    k = torch.randn(B, Hkv, N, d, device="cuda").to(torch.bfloat16)
    rot = fa.Rotary(torch.rand(width, device="cuda"))
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    for call in (fa.rope, fa.rope_backward):
        qo, ko = Guarded(q.shape, torch.bfloat16), Guarded(k.shape, torch.bfloat16)
        call(q, k, pos, rot, q_out=qo.t, k_out=ko.t)
        assert qo.intact() and ko.intact()
