"""The workspace of attention over a 4-bit cache (no GPU needed): a plan has one for either kind of cache, so those who use bf16
alone should not pay for more results than the 4-bit kernel's CTAs can leave."""

import ctypes

import pytest

from test_paged4_abi import fa  # noqa: F401
from test_paged_abi import _batch


def sizes(fa, **kw):  # noqa: F811
    b = ctypes.byref(_batch(fa, **kw))
    return fa.lib().fa_fwd_paged_workspace_bytes(b), fa.lib().fa_fwd_paged4_workspace_bytes(b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 32, 8), (8, 32, 8), (1, 64, 2), (32, 4, 4)])
def test_small_tiles_take_no_more_than_over_bf16(fa, d, max_q, Hq, Hkv):  # noqa: F811
    plain, four = sizes(fa, d=d, max_q=max_q, Hq=Hq, Hkv=Hkv)
    assert 0 < four <= plain


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q,Hq,Hkv", [(1, 16, 1), (4, 32, 8), (512, 32, 8), (300, 300, 1)])
def test_two_results_of_16_rows_for_each_cta(fa, d, max_q, Hq, Hkv):  # noqa: F811
    """9 to 16 rows, and those beside pairs: three CTAs per SM at d = 128, two at d = 64, on 160 SMs at most."""
    plain, four = sizes(fa, d=d, max_q=max_q, Hq=Hq, Hkv=Hkv)
    ctas = (3 if d == 128 else 2) * 160
    have = 2 * (2 if d == 128 else 3) * 160  # what the bf16 kernel's CTAs leave
    rows = 16 * (d + 3) * 4
    up = lambda n: (n + 255) // 256 * 256
    extra = up(2 * ctas * rows) + up(ctas * 20) - up(have * rows) - up(have // 2 * 20)
    assert four - plain == extra
