"""Weights of cached tokens: a table entry of -1 under a seen key is out of range like any other, and is reported."""

import math

import pytest
import torch

from gpu_util import fa_mod
from paged_util import assert_within, f64
from test_paged_weights_gpu import make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 64)])
@pytest.mark.parametrize("entry", [-1, -2, 1 << 30, -1 << 31])
def test_a_page_out_of_range_is_reported(fa, four, d, page, entry):
    lens = [(1, 400), (20, 300), (70, 500)]
    b = make(fa, four, lens, 4, 2, d, page, seed=page)
    plan = b.plan(fa)
    if four:
        _, lse = fa.forward_paged4(b.dev["q"], b.cache, plan)
    else:
        _, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan)
    fa.check()
    old = torch.rand(b.num_pages, 2, page, generator=torch.Generator().manual_seed(2))
    ref, tol, written = reference(b, lse, f64(old), True, 0, 1 / math.sqrt(d))
    for i, column in ((0, 3), (2, 1)):
        gone = int(b.table[i, column])
        b.dev["table"][i, column] = entry
        ref[gone] = f64(old)[gone]
        w = old.cuda()
        out = fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan, out=w.clone())
        with pytest.raises(fa.FAError) as e:
            fa.check()
        assert e.value.status == -8
        assert_within(out, ref, tol, "without the page")
        b.dev["table"][i, column] = gone
        ref, tol, written = reference(b, lse, f64(old), True, 0, 1 / math.sqrt(d))


@pytest.mark.parametrize("four", [False, True])
def test_entries_of_unseen_pages_may_be_anything(fa, four):
    """Before a window and behind the last key: -1 there is no error."""
    b = make(fa, four, [(1, 600), (3, 333)], 4, 2, 64, 16, seed=3)
    b.dev["table"][0, :20] = -1
    b.dev["table"][0, 38:] = -1
    b.dev["table"][1, 21:] = -1
    plan = b.plan(fa, window=100)
    lse = torch.full((4, 4), 5.0, device="cuda")
    w = torch.zeros(b.num_pages, 2, 16, device="cuda")
    fa.paged_weights(b.dev["q"], lse, b.cache if four else b.kc, w, plan)
    fa.check()
    ref, tol, _ = reference(b, lse, f64(torch.zeros_like(w)), True, 100, 0.125)
    assert_within(w, ref, tol, "weights")
