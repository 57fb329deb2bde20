"""Argument checks of the 4-bit cache, weight and eviction entry points that return before any CUDA call (no GPU needed)."""

import ctypes

import pytest

from test_paged_abi import BAD_BATCH, P, _batch, _cache, _ll, _rot

R = ctypes.byref


@pytest.fixture(scope="module")
def fa():
    from online_softmax_09_gb300 import build, fa

    build.build()
    fa.lib()
    return fa


def _cache4(fa, k=P, v=P, ks=P, vs=P, kst=(2048, 1024), vst=(2048, 1024), kss=(256, 128), vss=(256, 128), pages=10):
    return fa._Cache4(k, v, ks, vs, *kst, *vst, *kss, *vss, pages)


ST12 = (512, 128, 512, 128, 256, 128, 256, 128, 256, 128, 256, 128)


def _append(fa, q=None, qo=None, k=P, v=P, ko=None, vo=None, st=ST12, cache=None, batch=None, rotary=None, pos=None, pa=0):
    c, b = cache or _cache4(fa), batch or _batch(fa)
    return fa.lib().fa_paged_append4(q, qo, k, v, ko, vo, _ll(*st) if st else None, R(c), R(b),
                                     R(rotary) if rotary is not None else None, pos, pa, None)


def _forward(fa, q=P, st=(512, 128), cache=None, batch=None, o=P, lse=P, ws=P, n=1 << 32):
    c, b = cache or _cache4(fa), batch or _batch(fa)
    return fa.lib().fa_fwd_paged4(q, _ll(*st) if st else None, R(c), R(b), o, lse, 0.0, ws, n, None)


def _weights(fa, four, q=P, st=(512, 128), lse=P, cache=None, batch=None, w=P, out=P, ws=(32, 16, 32, 16)):
    c = cache or (_cache4(fa) if four else _cache(fa))
    b = batch or _batch(fa)
    fn = fa.lib().fa_paged_weights4 if four else fa.lib().fa_paged_weights
    return fn(q, _ll(*st) if st else None, lse, R(c), R(b), w, out, _ll(*ws) if ws else None, 0.0, None)


def _rows(fa, *rows):
    a = (fa._Rows * max(1, len(rows)))()
    for x, (base, strides, n) in zip(a, rows):
        x.base, x.bytes = base, n
        x.stride0, x.stride1, x.stride2 = strides
    return a


def _evict(fa, w=P, ws=(32, 16), rows=((P, (8192, 4096, 256), 256),), n=None, pages=10, batch=None, keep=P, max_keep=64, sinks=4,
           recent=8, to=P, stride=8, cols=4, kept=P, lens=P):
    b = batch or _batch(fa)
    return fa.lib().fa_paged_evict(w, _ll(*ws) if ws else None, _rows(fa, *rows), len(rows) if n is None else n, pages, R(b), keep,
                                   max_keep, sinks, recent, to, stride, cols, kept, lens, None)


def test_packed_rows_are_the_struct(fa):
    r = fa._Rows(P, 1, 2, 3, 4)
    assert fa._pack_rows(P, 1, 2, 3, 4) == bytes(r) and ctypes.sizeof(r) == 40
    assert ctypes.sizeof(fa._Cache4) == 104


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_batch_refusals(fa, kw, want):
    b = _batch(fa, **kw)
    assert _append(fa, batch=b) == want and _forward(fa, batch=b) == want
    assert _weights(fa, False, batch=b) == want and _weights(fa, True, batch=b) == want and _evict(fa, batch=b) == want


BAD_CACHE4 = [({"k": None}, -1), ({"v": None}, -1), ({"ks": None}, -1), ({"vs": None}, -1), ({"k": P + 8}, -3), ({"vs": P + 2}, -3),
              ({"pages": 0}, -1), ({"kst": (2048, 1032)}, -3), ({"vst": (0, 1024)}, -1), ({"kss": (256, -128)}, -1),
              ({"vss": (264, 128)}, -3), ({"kst": (1 << 32, 1024)}, -1)]


@pytest.mark.parametrize("kw,want", BAD_CACHE4)
def test_cache_refusals(fa, kw, want):
    c = _cache4(fa, **kw)
    assert _append(fa, cache=c) == want and _forward(fa, cache=c) == want
    if not any(n in kw for n in ("v", "vs", "vst", "vss")):
        assert _weights(fa, True, cache=c) == want


def test_append_refusals(fa):
    r = _rot(fa)
    assert _append(fa, k=None) == -1 and _append(fa, v=None) == -1 and _append(fa, st=None) == -1
    assert _append(fa, k=P + 8) == -3 and _append(fa, ko=P + 4) == -3 and _append(fa, vo=P + 2) == -3
    assert _append(fa, q=P, qo=P) == -1  # queries are only rotated
    assert _append(fa, q=P, rotary=r) == -1 and _append(fa, qo=P, rotary=r) == -1
    assert _append(fa, pos=P) == -1 and _append(fa, pos=P + 2, rotary=r) == -3 and _append(fa, pa=-1) == -1
    assert _append(fa, rotary=_rot(fa, axes=bytes([0, 1] * 32), naxes=2)) == -1
    assert _append(fa, st=ST12[:4] + (256, 4) + ST12[6:]) == -3
    assert _append(fa, ko=P, st=ST12[:8] + (0, 128, 256, 128)) == -1  # an output broadcast over tokens
    assert _append(fa, batch=_batch(fa, block_table=None)) == -1 and _append(fa, batch=_batch(fa, table_stride=-1)) == -1
    assert _append(fa, batch=_batch(fa, T=0)) == 0 and _append(fa, batch=_batch(fa, S=0)) == 0


def test_attention_refusals(fa):
    L, b = fa.lib(), _batch(fa)
    need = L.fa_fwd_paged4_workspace_bytes(R(b))
    assert need > 0 and L.fa_fwd_paged4_workspace_bytes(None) == 0
    for kw in ({"d": 96}, {"Hq": 3}, {"max_q": -1}):
        assert L.fa_fwd_paged4_workspace_bytes(R(_batch(fa, **kw))) == 0
    assert _forward(fa, n=need - 1) == -6 and _forward(fa, ws=None) == -6 and _forward(fa, ws=P + 8) == -3
    assert _forward(fa, q=None) == -1 and _forward(fa, o=None) == -1 and _forward(fa, lse=None) == -1 and _forward(fa, st=None) == -1
    assert _forward(fa, q=P + 8) == -3 and _forward(fa, o=P + 8) == -3 and _forward(fa, lse=P + 2) == -3
    assert _forward(fa, st=(512, 12)) == -3 and _forward(fa, st=(-512, 128)) == -1
    assert _forward(fa, q=P, o=P) == -1  # outputs over the queries
    assert _forward(fa, batch=_batch(fa, T=0)) == 0 and _forward(fa, batch=_batch(fa, S=0)) == 0


@pytest.mark.parametrize("four", [False, True])
def test_weight_refusals(fa, four):
    far = P + (1 << 20)
    assert _weights(fa, four, q=None) == -1 and _weights(fa, four, lse=None) == -1 and _weights(fa, four, st=None) == -1
    assert _weights(fa, four, w=None) == -1 and _weights(fa, four, out=None) == -1 and _weights(fa, four, ws=None) == -1
    assert _weights(fa, four, q=P + 8) == -3 and _weights(fa, four, lse=P + 2) == -3 and _weights(fa, four, w=P + 1) == -3
    assert _weights(fa, four, out=far, ws=(32, 16, 0, 16)) == -1 and _weights(fa, four, out=far, ws=(32, -16, 32, 16)) == -1
    assert _weights(fa, four, out=far, ws=(1 << 32, 16, 32, 16)) == -1
    assert _weights(fa, four, ws=(32, 16, 64, 16)) == -1  # in place, but at other strides
    assert _weights(fa, four, batch=_batch(fa, T=0)) == 0 and _weights(fa, four, batch=_batch(fa, S=0)) == 0
    assert _weights(fa, four, batch=_batch(fa, block_table=P + 2)) == -3


def test_evict_refusals(fa):
    assert _evict(fa, w=None) == -1 and _evict(fa, ws=None) == -1 and _evict(fa, keep=None) == -1 and _evict(fa, lens=None) == -1
    assert _evict(fa, kept=None) == -1 and _evict(fa, to=None) == -1 and _evict(fa, pages=0) == -1
    assert _evict(fa, w=P + 2) == -3 and _evict(fa, keep=P + 1) == -3 and _evict(fa, kept=P + 2) == -3 and _evict(fa, to=P + 3) == -3
    for kw in ({"max_keep": -1}, {"sinks": -1}, {"recent": -1}, {"stride": -1}, {"cols": -1}, {"n": 9}, {"n": -1}):
        assert _evict(fa, **kw) == -1
    assert _evict(fa, max_keep=65) == -1  # more than the other table's pages hold
    assert _evict(fa, rows=((None, (8192, 4096, 256), 256),)) == -1
    assert _evict(fa, rows=((P, (8192, 4096, 256), 0),)) == -1 and _evict(fa, rows=((P, (0, 4096, 256), 256),)) == -1
    assert _evict(fa, rows=((P, (8192, 4096, -256), 256),)) == -1
    assert _evict(fa, batch=_batch(fa, S=1 << 30), max_keep=64) in (-1, -6)
    assert _evict(fa, batch=_batch(fa, S=0)) == 0


def test_python_refuses_what_does_not_fit(fa):
    import torch

    x = torch.zeros(2, 1, 16, 32, dtype=torch.uint8)
    s = torch.zeros(2, 1, 16, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.PagedCache4(x, x, s, s)  # not on a GPU
    with pytest.raises(ValueError):
        fa.PagedCache4(x[0], x[0], s[0], s[0])
