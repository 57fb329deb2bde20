"""NaN in what a query sees makes its output NaN, whichever kernel takes it and however many CTAs share it."""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch, assert_within, attention_ref, f64

pytestmark = pytest.mark.gpu

# Pairs of tiles shared by many CTAs, one tile (halves at d = 64), small tiles joined by their last CTA or by a kernel.
LENS = [[(160, 6000)], [(40, 5000)], [(1, 6000)], [(6, 4000)], [(1, 700)] * 40, [(300, 500), (1, 900)]]


def _attend(b):
    fa = fa_mod()
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa))
    fa.check()
    return o, lse


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("cols", [2, 60000])
@pytest.mark.parametrize("d", [64, 128])
def test_a_query_with_nan(lens, cols, d):
    # All its scores are NaN, in every part of its keys; the other rows are as they were.
    b = Batch(lens, 2, 1, d, 16, seed=41, extra_cols=cols)
    row = b.cu[1] - 1
    b.dev["q"][row, 1, 3] = float("nan")
    o, lse = _attend(b)
    assert torch.isnan(o[row, 1].float()).all() and torch.isnan(lse[row, 1])
    o[row, 1], lse[row, 1] = 0, 0
    ql, n = lens[0]
    ro, rl, to, tl = attention_ref(f64(b.q[:ql]), f64(b.K[0]), f64(b.V[0]), n, True, 0, d ** -0.5, b.max_q)
    ro[row, 1], rl[row, 1] = 0, 0
    assert_within(o[:ql], ro, to, "o")
    assert_within(lse[:ql], rl, tl, "lse")


@pytest.mark.parametrize("lens", [x for x in LENS if x[0][1] >= 4000])
@pytest.mark.parametrize("d", [64, 128])
def test_a_run_of_keys_with_nan(lens, d):
    # Some CTAs' whole parts are NaN, others' are finite: no row that sees both is finite.
    b = Batch(lens, 2, 1, d, 16, seed=42)
    for x0 in range(0, 2000, 16):
        b.kc[int(b.table[0, x0 // 16])] = float("nan")
    o, lse = _attend(b)
    assert np.isnan(f64(o)).all() and np.isnan(f64(lse)).all()
