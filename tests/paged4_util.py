"""The 4-bit paged cache restated in NumPy, and batches over one (not collected as tests).

A group of 32 dims x: s = max|x| / 7 to four significant bits, u = 8 + x / s rounded, ties to even. In 64 bits both quotients
of bf16 numbers are exact enough to round as in exact arithmetic: one at a tie is a number of at most 9 bits, and any other
is off every tie by 2^-13 of itself or more (numerators and denominators have at most 12 bits between them). So codes and scales
have no tolerance.
"""

import numpy as np
import torch

from paged_util import Batch, f64

GROUP = 32


def quantise(x):
    """(codes [..., d] int, scales [..., d / 32], values [..., d]) of x [..., d] fp64."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.abs(g).max(-1)
        m, e = np.frexp(top / 7)
        s = np.ldexp(np.rint(m * 16), e - 4)
        bad = ~(top < 2.0 ** 120)  # NaN too
        none = top < 2.0 ** -100
        s = np.where(bad, np.nan, np.where(none, 0.0, s))
        u = np.where((bad | none)[..., None], 8, np.rint(g / np.where(none | bad, 1.0, s)[..., None]) + 8)
        u = np.where(np.isnan(u), 8, u)
        val = (u - 8) * s[..., None]
    return u.reshape(x.shape).astype(np.int64), s, val.reshape(x.shape)


def pack(u):
    """Codes [..., d] as bytes [..., d / 2]: word i holds dims 8 i .., dim 8 i + 2 j + e from bit 4 j + 16 e on."""
    w = np.zeros((*u.shape[:-1], u.shape[-1] // 8), dtype=np.uint32)
    for i in range(8):
        w |= u[..., i::8].astype(np.uint32) << np.uint32(4 * (i // 2) + 16 * (i % 2))
    return w.astype("<u4").view(np.uint8)


def unpack(b):
    w = np.ascontiguousarray(b).view("<u4")
    u = np.zeros((*w.shape[:-1], w.shape[-1] * 8), dtype=np.int64)
    for i in range(8):
        u[..., i::8] = (w >> np.uint32(4 * (i // 2) + 16 * (i % 2))) & 15
    return u


def values(codes, scales):
    """What codes [..., d / 2] and scales [..., d / 32] stand for, fp64."""
    return (unpack(codes) - 8) * np.repeat(np.asarray(scales, dtype=np.float64), GROUP, -1)


def cache_of(fa, kc, vc, apart=False):
    """A PagedCache4 of bf16 caches [pages, Hkv, page, d]; ``apart``: pages and heads at strides of their own."""
    parts = []
    for x in (kc, vc):
        u, s, _ = quantise(f64(x))
        parts.append((torch.from_numpy(pack(u)), torch.from_numpy(s).to(torch.bfloat16)))
    t = [parts[0][0], parts[1][0], parts[0][1], parts[1][1]]
    out = []
    for x in t:
        x = x.cuda()
        if apart:  # [Hkv][pages] order with a gap behind every page
            w = x.transpose(0, 1)
            big = torch.full((w.shape[0], w.shape[1], w.shape[2] + 16, w.shape[3]), 1, dtype=x.dtype, device="cuda")
            big[:, :, :w.shape[2]] = w
            x = big[:, :, :w.shape[2]].transpose(0, 1)
        out.append(x)
    return fa.PagedCache4(*out)


class Batch4(Batch):
    """A Batch over a 4-bit cache; K and V are the values that it stands for. Unseen slots hold scales of NaN."""

    def __init__(self, fa, *a, apart=False, **kw):
        super().__init__(*a, **kw)
        self.K = [torch.from_numpy(quantise(f64(x))[2]).to(torch.bfloat16) for x in self.K]
        self.V = [torch.from_numpy(quantise(f64(x))[2]).to(torch.bfloat16) for x in self.V]
        self.cache = cache_of(fa, self.kc.cpu(), self.vc.cpu(), apart)
        # The same values in bf16.
        self.kc, self.vc = (torch.from_numpy(quantise(f64(x))[2]).to(torch.bfloat16).cuda() for x in (self.kc, self.vc))
