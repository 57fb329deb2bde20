"""Windows up to the largest int over sequences with fewer cached tokens than new ones (fa_fwd_paged)."""

import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch

pytestmark = pytest.mark.gpu

FILL = -7.0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 40, 2 ** 30])
@pytest.mark.parametrize("lens", [[(5, 2), (1, 3), (4, 1), (6, 0)], [(40, 20), (300, 220), (2, 2), (150, 3)]])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_beyond_every_length(window, lens, d):
    # Positions before the first key are negative: the window's start lies below any int's range.
    fa = fa_mod()
    b = Batch(lens, 4, 2, d, 16, seed=61, pad=1)
    o = torch.full((b.T, b.Hq, d), FILL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.Hq), FILL, device="cuda")
    fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa, True, window), out=o, lse=lse)
    fa.check()
    b.check(o, lse, True, 0, None, FILL)
