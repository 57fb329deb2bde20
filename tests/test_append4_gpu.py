"""New tokens into a 4-bit paged cache: codes, scales and the values handed back, bit for bit where keys are not turned.

Turned keys: the kernel's bf16 key is within rope_ref's tolerance of the 64-bit one (paged_util.py), that is two neighbouring
bf16 numbers at most; a group's scale and codes have to be those of some key within it. With the group's magnitude off by
r = 2^-8 + 2^-19 relative at most, s may fall to the next of its steps, and a value is off by its own rounding:
|value - x| <= s / 2 + |x - x'|, s <= (17 / 16) (max|x| / 7) (1 + r).
"""

import numpy as np
import pytest
import torch

from gpu_util import fa_mod
from paged4_util import Batch4, pack, quantise, values
from paged_util import f64, rope_ref, rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return fa_mod()


def snapshot(c):
    return [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def places(b):
    """(token, sequence, position, page, slot) of every new token."""
    for i, (ql, n) in enumerate(b.lens):
        for j in range(ql):
            x = n - ql + j
            yield b.cu[i] + j, i, x, int(b.table[i, x // b.page]), x % b.page


def check_cache(b, before, want_k, want_v, k_out=None, v_out=None, exact_keys=True, key_tol=None):
    """The new tokens' slots hold want_k, want_v [T, Hkv, d] quantised; all other bytes are as before."""
    after = snapshot(b.cache)
    touched = torch.zeros(after[0].shape[:3], dtype=torch.bool)
    for name, want, codes, scales, out in (("k", want_k, after[0], after[2], k_out), ("v", want_v, after[1], after[3], v_out)):
        u, s, val = quantise(want)
        cc, sc = codes.cpu().numpy(), f64(scales)
        for t, _, _, page, slot in places(b):
            touched[page, :, slot] = True
            if name == "v" or exact_keys:
                np.testing.assert_array_equal(cc[page, :, slot], pack(u[t]))
                np.testing.assert_array_equal(sc[page, :, slot], s[t])
            got = values(cc[page, :, slot], sc[page, :, slot])
            if not (name == "v" or exact_keys):
                top = np.abs(want[t]).reshape(b.Hkv, -1, 32).max(-1)
                r = 2.0 ** -8 + 2.0 ** -19
                step = np.repeat(17 / 16 * top / 7 * (1 + r), 32, -1)
                assert np.all(np.abs(got - want[t]) <= step / 2 + key_tol[t])
            if out is not None:
                np.testing.assert_array_equal(f64(out[t]), got)
    touched = touched.cuda()
    for x, y in zip(before, after):
        assert same_bits(x[~touched], y[~touched])


def tokens(b, seed, wide=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(b.T, 2 * b.Hkv, b.d, generator=g)
    if wide:  # magnitudes from 2^-90 to 2^90, group by group
        x = x * torch.pow(2.0, torch.randint(-90, 90, (b.T, 2 * b.Hkv, b.d // 32), generator=g).float()).repeat_interleave(32, -1)
    x = x.to(torch.bfloat16)
    return x, x.cuda()


LENS = [(1, 1), (3, 40), (0, 9), (17, 17), (1, 33), (20, 70), (0, 0), (2, 128)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (8, 8), (10, 5)])
def test_keys_as_they_are(fa, d, page, Hq, Hkv):
    b = Batch4(fa, LENS, Hq, Hkv, d, page, seed=page, pad=2, lead=1, apart=Hkv == 5)
    x, dev = tokens(b, 5, wide=Hkv == 5)
    before = snapshot(b.cache)
    ko, vo = (torch.full((b.T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.paged_append4(None, dev[:, :Hkv], dev[:, Hkv:], b.cache, b.plan(fa), k_out=ko, v_out=vo)
    fa.check()
    check_cache(b, before, f64(x[:, :Hkv]), f64(x[:, Hkv:]), ko, vo)
    inside = torch.zeros(b.T, dtype=torch.bool)
    for t, *_ in places(b):
        inside[t] = True
    assert bool((ko[~inside.cuda()] == 7).all()) and bool((vo[~inside.cuda()] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
def test_ties_zeros_and_values_out_of_range(fa, d):
    b = Batch4(fa, [(6, 6)], 1, 1, d, 16, seed=1)
    x, _ = tokens(b, 1)
    x[0, 0] = 0
    x[1, 0, :32] = (torch.arange(32) - 16) * 0.5  # max 8: s rounds to 1.125
    x[2, 0, :32] = torch.arange(32) * (7 / 31) // 0.5 * 0.5  # max 7: s = 1, halves are ties
    x[2, 0, 31] = 7
    x[3, 0, 3] = float("inf")
    x[3, 1, 40] = float("nan")
    x[4, 0, 0] = 2.0 ** 120
    x[4, 1, 32:] = 2.0 ** -101
    x[5, 0, :32] = 119.0 * torch.sign(x[5, 0, :32].float())  # max / 7 = 17: between 16 and 18
    x[5, 1, :32] = 2.0 ** 119 * 1.9
    x = x.to(torch.bfloat16)
    before = snapshot(b.cache)
    ko, vo = (torch.empty(b.T, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.paged_append4(None, x[:, :1].cuda(), x[:, 1:].cuda(), b.cache, b.plan(fa), k_out=ko, v_out=vo)
    fa.check()
    check_cache(b, before, f64(x[:, :1]), f64(x[:, 1:]), ko, vo)


@pytest.mark.parametrize("d,rot,interleaved,axes", [(128, 128, False, 1), (64, 64, True, 1), (128, 48, False, 1),
                                                    (128, 64, True, 3), (64, 16, False, 2)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (40, 40)])
def test_turned_keys_and_queries(fa, d, rot, interleaved, axes, Hq, Hkv):
    b = Batch4(fa, LENS, Hq, Hkv, d, 32, seed=rot, pad=2, lead=1)
    x, dev = tokens(b, 7)
    ids = [i % axes for i in range(rot // 2)]
    freq = rotary(rot)
    R = fa.Rotary(freq.cuda(), interleaved=interleaved, axes=ids if axes > 1 else None)
    pos = torch.zeros(axes, b.T, dtype=torch.int32)
    for t, _, at, _, _ in places(b):
        pos[:, t] = at
    if axes > 1:
        pos[1:] = torch.randint(0, 5000, (axes - 1, b.T), generator=torch.Generator().manual_seed(3))
    before = snapshot(b.cache)
    ko, vo = (torch.full((b.T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = fa.paged_append4(b.dev["q"], dev[:, :Hkv], dev[:, Hkv:], b.cache, b.plan(fa), rotary=R,
                         positions=pos.cuda() if axes > 1 else None, k_out=ko, v_out=vo)
    fa.check()
    each = np.stack([pos[a].numpy() for a in ids], -1)[:, None]
    rk, tk = rope_ref(f64(x[:, :Hkv]), each, freq, interleaved)
    rq, tq = rope_ref(f64(b.q), each, freq, interleaved)
    check_cache(b, before, rk, f64(x[:, Hkv:]), ko, vo, exact_keys=False, key_tol=tk)
    for t, *_ in places(b):
        assert np.all(np.abs(f64(q[t]) - rq[t]) <= tq[t])


def test_turned_keys_are_those_of_the_bf16_cache(fa):
    """Keys are quantised from what fa_paged_append stores, bit for bit."""
    b = Batch4(fa, LENS, 4, 2, 128, 16, seed=9)
    x, dev = tokens(b, 9)
    R = fa.Rotary(rotary(128).cuda())
    plan = b.plan(fa)
    kc, vc = b.kc.clone(), b.vc.clone()
    q = fa.paged_append(b.dev["q"], dev[:, :2], dev[:, 2:], kc, vc, plan, R)
    before = snapshot(b.cache)
    q4 = fa.paged_append4(b.dev["q"], dev[:, :2], dev[:, 2:], b.cache, plan, R)
    fa.check()
    assert torch.equal(q, q4)
    kc, turned = kc.cpu(), np.zeros((b.T, 2, 128))
    for t, _, _, page, slot in places(b):
        turned[t] = f64(kc[page, :, slot])
    check_cache(b, before, turned, f64(x[:, 2:]))


def test_values_in_place_and_pages_out_of_range(fa):
    b = Batch4(fa, [(3, 20), (2, 40)], 2, 2, 64, 16, seed=4)
    x, dev = tokens(b, 4)
    b.dev["table"][1, 2] = b.num_pages  # positions 32 .. 47 of the second sequence
    before = snapshot(b.cache)
    fa.paged_append4(None, dev[:, :2], dev[:, 2:], b.cache, b.plan(fa), k_out=dev[:, :2], v_out=dev[:, 2:])
    with pytest.raises(fa.FAError) as e:
        fa.check()
    assert e.value.status == -8
    b.lens = [(3, 20), (0, 38)]
    check_cache(b, before, f64(x[:, :2]), f64(x[:, 2:]), dev[:, :2], dev[:, 2:])
    assert torch.equal(dev[3:].cpu(), x[3:])  # not stored, not written
