"""Outputs of fa_fwd_paged beside, between and in place of its queries."""

import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[(1, 100)], [(1, 100), (2, 40)], [(40, 100), (1, 60)]])
def test_outputs_next_to_queries(lens):
    fa = fa_mod()
    b = Batch(lens, 4, 2, 64, 16, seed=71)
    T, H, d = b.T, b.Hq, b.d
    plan = b.plan(fa)
    n = T * H * d
    for first in (0, n):  # queries before and behind the outputs, in one buffer
        buf = torch.zeros(2 * n, dtype=torch.bfloat16, device="cuda")
        q, o = buf[first:first + n].view(T, H, d), buf[n - first:2 * n - first].view(T, H, d)
        q.copy_(b.dev["q"])
        b.check(*fa.forward_paged(q, b.kc, b.vc, plan, out=o))
        fa.check()
    room = torch.zeros(H, 3 * T * H, d, dtype=torch.bfloat16, device="cuda")  # heads outermost, outputs in a gap
    q, o = room[:, :T].transpose(0, 1), room[1, T:T + T * H].view(T, H, d)
    q.copy_(b.dev["q"])
    b.check(*fa.forward_paged(q, b.kc, b.vc, plan, out=o))
    fa.check()


def test_outputs_over_queries_are_refused():
    fa = fa_mod()
    b = Batch([(1, 100), (40, 60)], 4, 2, 64, 16, seed=72)
    plan = b.plan(fa)
    q = b.dev["q"]
    with pytest.raises(fa.FAError) as e:
        fa.forward_paged(q, b.kc, b.vc, plan, out=q)
    assert e.value.status == -1
    buf = torch.zeros(b.T + 1, b.Hq, b.d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FAError):
        fa.forward_paged(buf[1:], b.kc, b.vc, plan, out=buf[:-1])
    fa.check()
