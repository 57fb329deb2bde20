"""Chunks over a 4-bit cache and over a bf16 cache of the same values, where the two are divided among CTAs or walked in orders
of their own: a table for contexts beyond L2, single tokens in the batch, more than 128 heads per kv head. Both stay within the
bounds of paged_util.py; that they have the same bits is not promised."""

import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv,cols", [([(300, 2000), (70, 900)], 4, 2, 600), ([(200, 700), (1, 2500), (1, 60), (90, 90)], 4, 2, 0),
                                              ([(20, 300), (1, 50)], 160, 1, 0)])
def test_both_kinds_of_cache(fa, d, lens, Hq, Hkv, cols):
    b = Batch4(fa, lens, Hq, Hkv, d, 256 if cols else 32, seed=d, extra_cols=cols + 2)
    plan = b.plan(fa)
    results = [fa.forward_paged4(b.dev["q"], b.cache, plan)]
    kc, vc = (torch.nan_to_num(x, nan=0.0) for x in (b.kc, b.vc))
    results.append(fa.forward_paged(b.dev["q"], kc, vc, plan))
    fa.check()
    for o, lse in results:
        b.check(o, lse)
