"""Sizes at which the eviction's counts would pass 32 bits are refused before any CUDA call (no GPU needed)."""

import pytest

from test_paged4_abi import _evict, fa  # noqa: F401
from test_paged_abi import _batch

MOST = 2 ** 31 - 2 ** 16 - 1  # as many tokens as a sequence may have


@pytest.mark.parametrize("max_keep", [MOST + 1, 2 ** 31 - 32, 2 ** 31 - 1])
def test_more_tokens_kept_than_a_sequence_can_have(fa, max_keep):  # noqa: F811
    assert _evict(fa, max_keep=max_keep, cols=1 << 28) == -1
    assert _evict(fa, max_keep=max_keep, cols=1 << 28, batch=_batch(fa, S=0)) == -1


def test_python_refuses_them_before_it_allocates(fa):  # noqa: F811
    with pytest.raises(ValueError):
        fa._check_keep(MOST + 1, 0, 0)
    with pytest.raises(ValueError):
        fa._check_keep(-1, 0, 0)
    assert fa._check_keep(MOST, 2 ** 31 - 1, 2 ** 31 - 1) == (MOST, 2 ** 31 - 1, 2 ** 31 - 1)
