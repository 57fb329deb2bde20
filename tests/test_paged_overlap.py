"""fa_fwd_paged refuses outputs that share memory with its queries (before any CUDA call: no GPU needed)."""

import ctypes

import pytest

from test_paged_abi import P, _batch, _cache, _ll, fa  # noqa: F401

ROW = 128 * 2  # bytes of a head of one token


# o against q at P: 4 tokens of 4 heads, token stride 512 elements (dense), 1024 (every other row), or heads outermost.
@pytest.mark.parametrize("strides,at", [
    ((512, 128), 0), ((512, 128), 16), ((512, 128), 16 * ROW - 16), ((512, 128), -16 * ROW + 16),
    ((1024, 128), 4 * ROW), ((1024, 128), 28 * ROW - 16), ((128, 512), 0), ((128, 512), 16 * ROW - 16),
    ((1 << 20, 128), (3 << 21) - 16 * ROW + 16), ((128, 1 << 20), (1 << 21) + 4 * ROW - 16), ((512, 128), -16)])
def test_overlapping_outputs(fa, strides, at):  # noqa: F811
    L, b, c = fa.lib(), _batch(fa), _cache(fa)
    q = 1 << 30
    assert L.fa_fwd_paged(q, _ll(*strides), ctypes.byref(c), ctypes.byref(b), q + at, P, 0.0, P, 1 << 30, None) == -1


def test_one_token_in_place(fa):  # noqa: F811
    L, b, c = fa.lib(), _batch(fa, T=1, Hq=4), _cache(fa)
    for at in (0, 3 * ROW, -3 * ROW):
        assert L.fa_fwd_paged(1 << 30, _ll(0, 128), ctypes.byref(c), ctypes.byref(b), (1 << 30) + at, P, 0.0, P, 1 << 30,
                              None) == -1
