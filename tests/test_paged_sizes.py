"""Sizes that do not fit the C ABI's ints are refused, not cut off (no GPU needed)."""

import pytest
import torch

from test_paged_abi import fa  # noqa: F401

NAMES = ("S", "T", "max_q", "max_pages", "page_size", "Hq", "Hkv", "d", "causal", "window")
GOOD = dict(S=2, T=4, max_q=2, max_pages=8, page_size=16, Hq=4, Hkv=2, d=128, causal=1, window=0)


@pytest.mark.parametrize("name", ["T", "max_q", "max_pages", "page_size", "Hq", "Hkv", "d", "window"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 16, 2 ** 63 - 1, -2 ** 31 - 1, -2 ** 32 + 16])
def test_sizes_beyond_an_int(fa, name, value):  # noqa: F811
    args = dict(GOOD, **{name: value})
    with pytest.raises(ValueError):
        fa.PagedPlan(*[args[n] for n in NAMES], torch.device("cuda", 0), None)
