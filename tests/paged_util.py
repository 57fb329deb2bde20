"""fp64 references and batches for the rotary and paged-cache tests (not collected as tests).

Tolerances, derived from the kernels' arithmetic (bf16 half step: 2^-8 relative; fp32: 2^-24):

rotation: y = a cos + b sin is formed in fp32 from bf16 a, b and rounded to bf16 once. The angle is off by
  half a float step of at most half a turn (9.4e-8 rad); cos and sin by two float steps (2.4e-7); two products and a
  sum by 3 * 2^-24. So |y - ref| <= 2^-8 |ref| + 6e-7 (|a| + |b|). (The angle is off by 2^-52.3 of itself as well,
  3.4e-7 rad at position 2^31: not counted, and inside what the other parts leave of their bounds.)

attention: a score is off by e_s = 2 d 2^-24 scale sum|q k| (fp32 accumulation in any order, truncating), its
  weight therefore by 2 e_s + 2^-20 (exp2 and the reference's rescales), and by 2^-8 once rounded for the product
  with V. o is the weighted mean under the rounded weights, so with eps = 2^-8 + 2 e_s + 2^-20 and weights p:
  |o - ref| <= 1.02 eps sum_j p_j |v_j - ref| + 2^-8 |ref| + 2^-20 max|v|  (fp32 sums of the products: the last).
  So it is in the tiles of 16 or 32 rows, whose rounded weights are summed. The pairs of 128-row tiles (sequences of
  more than 32 rows, new tokens times heads per kv head; at d = 128 of more than 16, if the batch's limit of new tokens
  allows more than 32) divide
  by the sum of the weights before rounding, plus the rounding of each block's largest one: with p'_j = p_j (1 + d_j),
  |d_j| <= 2^-8, and M the blocks' largest,
      o' - ref = sum_j p_j d_j v_j - ref sum_{j in M} p_j d_j  (to first order),
  whose size is at most 2^-8 (sum_j p_j |v_j| + |ref|), since sum_M p_j <= 1. A score's error still moves numerator and
  denominator alike. So there
  |o - ref| <= 1.02 (2^-8 (sum_j p_j |v_j| + |ref|) + (2 e_s + 2^-20) sum_j p_j |v_j - ref|) + 2^-8 |ref| + 2^-20 max|v|.
  lse: e_s + 2^-20 + (n / 64 + 16) 2^-24 + 2^-22 |lse|.
"""

import math

import numpy as np
import torch

BF = 2.0 ** -8


def rotary(rot, theta=1.0e4):
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    return (theta ** (-i / rot)).to(torch.float32)


def rope_ref(x, pos, inv_freq, interleaved=False, inverse=False):
    """x [..., d] and pos [..., rot / 2] (each pair's position) to (rotated, tolerance), fp64."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(inv_freq, dtype=np.float64)
    rot = 2 * w.size
    phi = np.asarray(pos, dtype=np.float64) * w * (-1 if inverse else 1)
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2),
                                                                              np.arange(rot // 2, rot))
    a, b = x[..., ia], x[..., ib]
    y, tol = x.copy(), np.zeros_like(x)
    y[..., ia] = a * np.cos(phi) - b * np.sin(phi)
    y[..., ib] = b * np.cos(phi) + a * np.sin(phi)
    mag = np.abs(a) + np.abs(b)
    tol[..., ia] = BF * np.abs(y[..., ia]) + 6e-7 * mag
    tol[..., ib] = BF * np.abs(y[..., ib]) + 6e-7 * mag
    return y, tol


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def assert_within(got, ref, tol, what=""):
    got = f64(got) if torch.is_tensor(got) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - ref) <= tol))
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]} for {ref[i]} "
                             f"(tolerance {np.broadcast_to(tol, bad.shape)[i]})")


def attention_ref(q, K, V, n, causal, window, scale, max_q=None):
    """One sequence: q [ql, Hq, d], K, V [n, Hkv, d] fp64 -> o, lse and their tolerances."""
    ql, Hq, d = q.shape
    G = Hq // K.shape[1] if n else 1
    pairs = G <= 128 and ql * G > (16 if d == 128 and (max_q or ql) * G > 32 else 32)
    o = np.zeros((ql, Hq, d))
    lse = np.full((ql, Hq), -np.inf)
    to, tl = np.zeros((ql, Hq, d)), np.zeros((ql, Hq))
    for j in range(ql):
        p = n - ql + j
        hi = min(n, p + 1) if causal else n
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            k, v = K[lo:hi, h // G], V[lo:hi, h // G]
            x = scale * (k @ q[j, h])
            es = 2 * d * 2.0 ** -24 * scale * float(np.max(np.abs(k) @ np.abs(q[j, h])))
            m = x.max()
            e = np.exp(x - m)
            s = e.sum()
            w = e / s
            o[j, h] = w @ v
            lse[j, h] = m + math.log(s)
            spread = w @ np.abs(v - o[j, h])
            rounding = w @ np.abs(v) + np.abs(o[j, h]) if pairs else spread
            to[j, h] = 1.02 * (BF * rounding + (2 * es + 2.0 ** -20) * spread) + BF * np.abs(o[j, h])
            to[j, h] += 2.0 ** -20 * np.abs(v).max()
            tl[j, h] = es + 2.0 ** -20 + ((hi - lo) / 64 + 16) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[j, h])
    return o, lse, to, tl


class Batch:
    """A ragged batch: lens [(new, cached)], a page table over shuffled pages, everything past a sequence's cached
    tokens set to NaN or to numbers out of range (what stands before a window is finite)."""

    def __init__(self, lens, Hq, Hkv, d, page, seed=0, layout="phsd", pad=0, lead=0, poison=True, extra_cols=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.page = lens, Hq, Hkv, d, page
        pages = [(n + page - 1) // page for _, n in lens]
        self.num_pages = sum(pages) + 2
        order = torch.randperm(self.num_pages, generator=g).tolist()
        cols = max(pages + [1]) + extra_cols
        self.table = torch.full((len(lens), cols), -7 if poison else 0, dtype=torch.int32)
        self.table[:, 1::2] = 1 << 30 if poison else 0
        kc = torch.full((self.num_pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16)
        vc = torch.full((self.num_pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16)
        vc[:, :, ::2] = float("inf")
        self.K, self.V = [], []
        at = 0
        for i, (_, n) in enumerate(lens):
            ids = order[at:at + pages[i]]
            at += pages[i]
            self.table[i, :pages[i]] = torch.tensor(ids, dtype=torch.int32)
            K = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
            V = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
            for x in range(n):
                kc[ids[x // page], :, x % page] = K[x]
                vc[ids[x // page], :, x % page] = V[x]
            self.K.append(K)
            self.V.append(V)
        cu = [lead]
        for ql, _ in lens:
            cu.append(cu[-1] + ql)
        self.T = cu[-1] + pad
        self.cu = cu
        self.q = torch.randn(self.T, Hq, d, generator=g).to(torch.bfloat16)
        self.cu_q = torch.tensor(cu, dtype=torch.int32)
        self.kv_lens = torch.tensor([n for _, n in lens], dtype=torch.int32)
        self.max_q = max([ql for ql, _ in lens] + [0])
        if layout == "phsd":
            self.kc, self.vc = kc.cuda(), vc.cuda()
        elif layout == "pshd":
            self.kc, self.vc = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (kc, vc))
        else:  # both in one tensor
            both = torch.stack([kc, vc], 1).cuda()
            self.kc, self.vc = both[:, 0], both[:, 1]
        self.dev = {"q": self.q.cuda(), "cu_q": self.cu_q.cuda(), "kv_lens": self.kv_lens.cuda(),
                    "table": self.table.cuda()}

    def plan(self, fa, causal=True, window=0, **kw):
        D = self.dev
        return fa.paged_plan(D["cu_q"], D["kv_lens"], D["table"], num_tokens=self.T, max_q=self.max_q,
                             page_size=self.page, Hq=self.Hq, Hkv=self.Hkv, d=self.d, causal=causal, window=window, **kw)

    def check(self, o, lse, causal=True, window=0, scale=None, fill=None):
        """o, lse against the reference; rows of no sequence still hold ``fill``."""
        scale = scale or 1 / math.sqrt(self.d)
        o, lse = f64(o), f64(lse)
        inside = np.zeros(self.T, dtype=bool)
        for i, (ql, n) in enumerate(self.lens):
            a = self.cu[i]
            inside[a:a + ql] = True
            ro, rl, to, tl = attention_ref(f64(self.q[a:a + ql]), f64(self.K[i]), f64(self.V[i]), n,
                                           causal or window > 0, window, scale, self.max_q)
            assert_within(lse[a:a + ql], rl, tl, f"lse of sequence {i} {self.lens[i]}")
            assert_within(o[a:a + ql], ro, to, f"o of sequence {i} {self.lens[i]}")
        if fill is not None:
            assert np.all(o[~inside] == fill) and np.all(lse[~inside] == fill)
