"""Argument checks of the rotary and paged entry points that return before any CUDA call (no GPU needed)."""

import ctypes

import pytest

P = 0x1000  # an aligned address that nothing may touch


@pytest.fixture(scope="module")
def fa():
    from online_softmax_09_gb300 import build, fa

    build.build()
    fa.lib()
    return fa


def _ll(*v):
    return (ctypes.c_longlong * len(v))(*v)


def test_packed_cache_is_the_struct(fa):
    c = fa._Cache(*range(1, 10))
    assert fa._pack_cache(*range(1, 10)) == bytes(c) and ctypes.sizeof(c) == 72


def _rot(fa, rot=128, axes=None, naxes=1, inv=P):
    return fa._Rotary(inv, axes, naxes, rot, 0)


def _rope(fa, q=P, qo=P, k=P, ko=P, strides=None, pos=P, pa=0, pb=0, rotary="ok", B=1, Hq=2, Hkv=1, N=4, d=128):
    r = _rot(fa) if rotary == "ok" else rotary
    s = _ll(*([1024, 512, 128] * 4)) if strides is None else strides
    out = set()
    for fn in (fa.lib().fa_rope, fa.lib().fa_rope_bwd):
        out.add(fn(q, qo, k, ko, s, pos, pa, pb, ctypes.byref(r) if r is not None else None, B, Hq, Hkv, N, d, None))
    assert len(out) == 1
    return out.pop()


def test_rope_refusals(fa):
    assert _rope(fa, q=None) == -1 and _rope(fa, qo=None) == -1
    assert _rope(fa, k=None) == -1 and _rope(fa, ko=None) == -1  # one without the other
    assert _rope(fa, q=P + 8) == -3 and _rope(fa, ko=P + 2) == -3 and _rope(fa, pos=P + 2) == -3
    assert _rope(fa, pos=None) == -1 and _rope(fa, rotary=None) == -1
    assert _rope(fa, B=0) == -1 and _rope(fa, N=0) == -1 and _rope(fa, Hq=0) == -1 and _rope(fa, Hkv=0) == -1
    assert _rope(fa, B=1 << 16, N=1 << 15) == -1  # too many tokens
    assert _rope(fa, d=96) == -2 and _rope(fa, d=256) == -2
    assert _rope(fa, strides=_ll(*([1024, 512, 128] * 3 + [1024, 512, 4]))) == -3
    assert _rope(fa, strides=_ll(*([1024, 512, 128] * 3 + [1024, 512, 0]))) == -1  # an output broadcast over tokens
    assert _rope(fa, B=2, strides=_ll(*([-1024, 512, 128] + [1024, 512, 128] * 3))) == -1
    assert _rope(fa, strides=_ll(*([1024, -512, 128] + [1024, 512, 128] * 3))) == -1
    assert _rope(fa, pa=-1) == -1 and _rope(fa, pb=-1) == -1
    for bad in (_rot(fa, rot=0), _rot(fa, rot=8), _rot(fa, rot=40), _rot(fa, rot=256), _rot(fa, naxes=0),
                _rot(fa, naxes=5), _rot(fa, inv=None), _rot(fa, axes=bytes([1] * 64), naxes=1),
                _rot(fa, axes=bytes([0] * 63 + [3]), naxes=3)):
        assert _rope(fa, rotary=bad) == -1
    assert _rope(fa, rotary=_rot(fa, inv=P + 1)) == -3
    assert _rope(fa, rotary=_rot(fa, rot=128), d=64) == -1


def _batch(fa, **kw):
    b = dict(block_table=P, table_stride=8, plan=P, plan_bytes=1 << 30, S=2, T=4, max_q=2, max_pages=8, page_size=16,
             Hq=4, Hkv=2, d=128, causal=1, window=0)
    b.update(kw)
    return fa._Batch(*[b[n] for n, _ in fa._Batch._fields_])


def _cache(fa, k=P, v=P, ks=(4096, 2048, 128), vs=(4096, 2048, 128), pages=10):
    return fa._Cache(k, v, *ks, *vs, pages)


BAD_BATCH = [({"S": -1}, -1), ({"T": -1}, -1), ({"max_q": -1}, -1), ({"max_pages": 0}, -1), ({"window": -1}, -1),
             ({"max_q": 1 << 30}, -1), ({"T": (1 << 31) - 1}, -1), ({"max_pages": (1 << 27) - 1}, -1), ({"Hq": 0}, -1), ({"Hkv": 0}, -1), ({"Hq": 3}, -1), ({"d": 96}, -2), ({"page_size": 8}, -2),
             ({"page_size": 48}, -2), ({"page_size": 512}, -2), ({"max_pages": 1 << 28}, -1), ({"plan": None}, -6),
             ({"plan_bytes": 64}, -6), ({"plan": P + 8}, -3)]


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_batch_refusals(fa, kw, want):
    L, b, c = fa.lib(), _batch(fa, **kw), _cache(fa)
    st = _ll(512, 128, 512, 128, 256, 128, 256, 128)
    assert L.fa_paged_plan(P, P, ctypes.byref(b), None) == want
    assert L.fa_paged_append(None, None, P, P, st, ctypes.byref(c), ctypes.byref(b), None, None, 0, None) == want
    assert L.fa_fwd_paged(P, st, ctypes.byref(c), ctypes.byref(b), P, P, 0.0, P, 1 << 30, None) == want


def test_plan_refusals_and_sizes(fa):
    L = fa.lib()
    b = _batch(fa)
    assert L.fa_paged_plan(None, P, ctypes.byref(b), None) == -1
    assert L.fa_paged_plan(P, None, ctypes.byref(b), None) == -1
    assert L.fa_paged_plan(P, P + 1, ctypes.byref(b), None) == -3
    assert L.fa_paged_plan(P, P, None, None) == -1
    assert L.fa_paged_plan_bytes(-1) == 0 and L.fa_paged_plan_bytes(0) > 0
    assert L.fa_paged_plan_bytes(1000) > L.fa_paged_plan_bytes(10)
    short = _batch(fa, S=1000, plan_bytes=L.fa_paged_plan_bytes(1000) - 1)
    assert L.fa_paged_plan(P, P, ctypes.byref(short), None) == -6
    ws = lambda **kw: L.fa_fwd_paged_workspace_bytes(ctypes.byref(_batch(fa, **kw)))
    assert ws(d=96) == 0 and ws(Hq=3) == 0 and ws(max_q=-1) == 0 and L.fa_fwd_paged_workspace_bytes(None) == 0
    assert ws(d=128) > ws(d=64) > 0
    assert ws(max_q=100) > ws(max_q=1)  # chunks need room for larger partial results


BAD_CACHE = [({"k": None}, -1), ({"v": None}, -1), ({"k": P + 8}, -3), ({"v": P + 2}, -3), ({"pages": 0}, -1),
             ({"ks": (4096, 2048, 4)}, -3), ({"vs": (4096, -2048, 128)}, -1)]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_cache_refusals(fa, kw, want):
    L, b, c = fa.lib(), _batch(fa), _cache(fa, **kw)
    st = _ll(512, 128, 512, 128, 256, 128, 256, 128)
    assert L.fa_paged_append(None, None, P, P, st, ctypes.byref(c), ctypes.byref(b), None, None, 0, None) == want
    assert L.fa_fwd_paged(P, st, ctypes.byref(c), ctypes.byref(b), P, P, 0.0, P, 1 << 30, None) == want


def test_append_refusals(fa):
    L, b, c, r = fa.lib(), _batch(fa), _cache(fa), _rot(fa)

    def call(q=P, qo=P, k=P, v=P, st=(512, 128, 512, 128, 256, 128, 256, 128), cache=c, batch=b, rotary=r, pos=None,
             pa=0):
        return L.fa_paged_append(q, qo, k, v, _ll(*st), ctypes.byref(cache), ctypes.byref(batch),
                                 ctypes.byref(rotary) if rotary is not None else None, pos, pa, None)

    assert call(k=None) == -1 and call(v=None) == -1 and call(q=None) == -1 and call(qo=None) == -1
    assert call(q=P + 8) == -3 and call(v=P + 4) == -3 and call(pos=P + 2) == -3
    assert call(rotary=None) == -1  # queries are only rotated
    assert call(q=None, qo=None, rotary=None, pos=P) == -1
    assert call(rotary=_rot(fa, axes=bytes([0, 1] * 32), naxes=2)) == -1  # several axes need positions
    assert call(st=(512, 128, 0, 128, 256, 128, 256, 128)) == -1
    assert call(st=(512, 128, 512, 128, 256, 4, 256, 128)) == -3
    assert call(cache=_cache(fa, ks=(0, 2048, 128))) == -1  # all pages in one place
    assert call(pa=-1) == -1
    assert call(batch=_batch(fa, block_table=None)) == -1
    assert call(batch=_batch(fa, block_table=P + 2)) == -3
    assert call(batch=_batch(fa, table_stride=-1)) == -1
    assert call(batch=_batch(fa, T=0)) == 0 and call(batch=_batch(fa, S=0)) == 0  # nothing to do


def test_attention_refusals(fa):
    L, b, c = fa.lib(), _batch(fa), _cache(fa)
    need = L.fa_fwd_paged_workspace_bytes(ctypes.byref(b))

    def call(q=P, st=(512, 128), cache=c, batch=b, o=P, lse=P, ws=P, n=need):
        return L.fa_fwd_paged(q, _ll(*st) if st else None, ctypes.byref(cache), ctypes.byref(batch), o, lse, 0.0, ws, n,
                              None)

    assert call(q=None) == -1 and call(o=None) == -1 and call(lse=None) == -1 and call(st=None) == -1
    assert call(q=P + 8) == -3 and call(o=P + 8) == -3 and call(lse=P + 2) == -3 and call(ws=P + 8) == -3
    assert call(ws=None) == -6 and call(n=need - 1) == -6
    assert call(st=(512, 12)) == -3 and call(st=(-512, 128)) == -1
    assert call(batch=_batch(fa, block_table=None)) == -1
    assert call(batch=_batch(fa, T=0)) == 0 and call(batch=_batch(fa, S=0)) == 0


def test_python_refuses_cpu_tensors_and_wrong_shapes(fa):
    import torch

    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.Rotary(torch.ones(32))
    with pytest.raises(ValueError):
        fa.rope(x[0], None, torch.zeros(4, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        fa.rope(x, None, torch.zeros(4, dtype=torch.int32), None)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_plan(i, i[:1], i[None], 1, 1, 16, 2, 1, 64)
    assert fa.strerror(-8) != "unknown status"
