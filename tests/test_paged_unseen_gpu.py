"""Windowed attention over a paged cache whose slots before the window hold NaN and infinities (fa_fwd_paged).

What no query of a sequence sees may hold anything: the slots before the first new token's window, and the table
entries of pages that lie wholly before it. ``Batch`` fills every slot of a sequence; here those are taken back.
"""

import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch

pytestmark = pytest.mark.gpu

FILL = -7.0


def _hide_before_window(b, window):
    """Every slot that no query of its sequence sees set to NaN or infinity, every table entry for such slots alone to
    a number out of range; how many sequences' first visible key stands inside a page."""
    inside = 0
    for i, (ql, n) in enumerate(b.lens):
        lo = max(0, n - ql - window + 1) if ql else n
        for x0 in range(0, lo, b.page):
            page = int(b.table[i, x0 // b.page])
            for kind, value in ((0, float("nan")), (1, float("inf")), (2, -float("inf"))):
                slots = slice(kind, min(b.page, lo - x0), 3)
                b.kc[page, :, slots] = value
                b.vc[page, :, slots] = value
            if x0 + b.page <= lo:
                b.dev["table"][i, x0 // b.page] = -5 if x0 % (2 * b.page) else 1 << 29
        inside += lo % b.page > 0
    return inside


def _run(b, window, causal=True):
    fa = fa_mod()
    assert _hide_before_window(b, window) > 0
    out = []
    for _ in range(2):
        o = torch.full((b.T, b.Hq, b.d), FILL, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.T, b.Hq), FILL, device="cuda")
        fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa, causal, window), out=o, lse=lse)
        fa.check()
        out.append((o, lse))
    b.check(*out[0], causal, window, None, FILL)
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window", [1, 37, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks(page, window, d):
    # One tile (halves at d = 64), two tiles, several pairs; the first visible key at many places of its box.
    lens = [(40, 300), (33, 290), (90, 700), (150, 555), (257, 901), (64, 64), (100, 1230)]
    _run(Batch(lens, 4, 2, d, page, seed=page + window, pad=2), window)


@pytest.mark.parametrize("window", [1, 37, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_single_and_drafted_tokens(window, d):
    _run(Batch([(1, 300), (1, 77), (1, 1000), (1, 255)], 8, 2, d, 32, seed=window), window)
    _run(Batch([(4, 300), (7, 777), (2, 1000), (1, 255)], 8, 2, d, 64, seed=window + 1), window, causal=False)


@pytest.mark.parametrize("heads", [(6, 2), (16, 1), (3, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_beside_single_tokens(heads, d):
    _run(Batch([(1, 500), (60, 811), (1, 90), (0, 70), (9, 333), (130, 1000)], *heads, d, 128, seed=heads[0]), 150)


@pytest.mark.parametrize("lens,window", [([(40, 6000)], 3007), ([(160, 5000)], 2700), ([(300, 4000), (50, 3000)], 1500)])
@pytest.mark.parametrize("cols", [2, 40000])
@pytest.mark.parametrize("d", [64, 128])
def test_window_over_many_ctas(lens, window, cols, d):
    # Tiles that many CTAs share: the one with the first visible key; and the turned order of blocks (wide tables).
    _run(Batch(lens, 4, 1, d, 16, seed=window, extra_cols=cols), window)
