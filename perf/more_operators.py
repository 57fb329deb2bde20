"""Cases, plain forms and 64-bit definitions of the 4-bit paged cache, the attention over it, and eviction by weight.

Every case is a dict of plain values; ``prepare`` makes what a user's program holds before the call, ``run`` is one pass
(elementary torch operations in fp32 where ``own`` is false, the library's entry points where it is true) and ``exact``
the same outputs in 64 bits.

A 4-bit cache holds groups of 32 dims of a key or value: a scale, bf16 with four significant bits (the nearest to the
group's largest magnitude / 7), and a code 1..15 per dim, nearest to value / scale + 8 (ties to even both times). The 32-bit
word i of a group holds dims 8 i .. 8 i + 7, dim 8 i + 2 j + e in the bits from 4 j + 16 e on.
"""

import math
import random

import torch

own = False

HBM = 6.7e12  # bytes/s and flop/s used only to compare the cost of drawn cases with the listed ones
MMA = 1.9e15
GROUP = 32


# ---------------------------------------------------------------------------------------------------------- cases
def _case(name, op, S, q_min, q_max, kv_min, kv_max, Hq, Hkv, d, page, lens, **more):
    return {"name": name, "op": op, "S": S, "q_min": q_min, "q_max": q_max, "kv_min": kv_min, "kv_max": kv_max, "Hq": Hq,
            "Hkv": Hkv, "d": d, "page": page, "lens": lens, **more}


def listed():
    return [
        # One new token's keys and values of one conversation into the cache: latency.
        _case("append4-one-token", "append4", 1, 1, 1, 1000, 1000, 32, 8, 128, 16, 1),
        # A decode step of 64 conversations.
        _case("append4-decode-s64", "append4", 64, 1, 1, 100, 2000, 32, 8, 128, 16, 2),
        # Prompts of ragged lengths brought into the cache together.
        _case("append4-prompts-s8", "append4", 8, 300, 1900, 1900, 2500, 32, 8, 128, 64, 3),
        # One new token of one conversation of about a thousand tokens: latency.
        _case("attn4-one-token-kv1000", "attn4", 1, 1, 1, 1000, 1000, 32, 8, 128, 16, 4, window=0),
        # A decode step of 64 conversations of ragged lengths.
        _case("attn4-decode-s64", "attn4", 64, 1, 1, 200, 8192, 32, 8, 128, 16, 5, window=0),
        # Four drafted tokens checked for each of 48 conversations, d = 64, a sliding window.
        _case("attn4-draft4-s48-window", "attn4", 48, 4, 4, 500, 6000, 16, 4, 64, 32, 6, window=1024),
        # Two conversations as long as the long-context benchmark, one token each.
        _case("attn4-long-s2-kv131072", "attn4", 2, 1, 1, 120001, 131072, 32, 8, 128, 64, 7, window=0),
        # The next chunk of one long prompt.
        _case("attn4-chunk512-kv32768", "attn4", 1, 512, 512, 32768, 32768, 32, 8, 128, 64, 8, window=0),
        # The weights that a decode step gives to its cached tokens, added to what earlier steps gave.
        _case("weights-decode-s64", "weights", 64, 1, 1, 200, 8192, 32, 8, 128, 16, 9, window=0, bits=16),
        # The weights that the last 32 tokens of prompts give to all of them, over 4-bit keys, d = 64.
        _case("weights-last32-s8-4bit", "weights", 8, 32, 32, 4001, 16000, 16, 16, 64, 32, 10, window=0, bits=4),
        # Half the tokens of 32 short conversations are dropped, d = 64.
        _case("evict-s32-keep500", "evict", 32, 1, 1, 700, 1501, 16, 4, 64, 16, 11, keep=500, sinks=4, recent=64),
        # A long prompt cut down to an eighth.
        _case("evict-one-kv32768-keep4096", "evict", 1, 1, 1, 32768, 32768, 32, 8, 128, 64, 12, keep=4096, sinks=4,
              recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: each operator alike often, sizes log-uniform over the listed range, at most the largest listed cost."""
    cap = max(_cost(c) for c in listed())
    op = rng.choice(["append4", "attn4", "attn4", "weights", "evict"])
    while True:
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 5, 8, 16])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        S, lens = _log(rng, 1, 128), rng.randint(0, 10 ** 6)
        if op == "append4":
            q_max = rng.choice([1, 1, _log(rng, 2, 4096)])
            kv_max = q_max + _log(rng, 1, 4096)
            c = _case(None, op, S, rng.choice([1, q_max]), q_max, q_max, kv_max, Hkv * G, Hkv, d, page, lens)
        elif op == "evict":
            kv_max = _log(rng, 16, 131072)
            c = _case(None, op, S, 1, 1, _log(rng, 1, kv_max), kv_max, Hkv * G, Hkv, d, page, lens,
                      keep=_log(rng, 1, kv_max), sinks=rng.choice([0, 1, 4, 17]), recent=rng.choice([0, 1, 64, 200]))
        else:
            q_max = rng.choice([1, 1, _log(rng, 2, 1024)])
            kv_max = max(q_max, _log(rng, 16, 131072))
            c = _case(None, op, S, rng.choice([1, q_max]), q_max, max(q_max, _log(rng, 1, kv_max)), kv_max, Hkv * G, Hkv, d,
                      page, lens, window=rng.choice([0, 0, _log(rng, 16, 8192)]))
            if op == "weights":
                c["bits"] = rng.choice([16, 4])
        kv = max(n for _, n in _lengths(c))
        # (The plain forms fill all sequences up to the longest.)
        if S * kv * Hkv * d <= 2 ** 29 and S * c["q_max"] * Hkv * G * kv <= 2 ** 29 and _cost(c) <= cap:
            del c["name"]
            return c


def _lengths(c):
    """(new tokens, cached tokens with them) of every sequence; the case alone decides."""
    r = random.Random(c["lens"])
    return [(r.randint(c["q_min"], c["q_max"]), r.randint(c["kv_min"], c["kv_max"])) for _ in range(c["S"])]


def _pairs(q, n, window):
    """Visible (query token, key) pairs and the number of keys that any of the q last queries of n positions sees."""
    lo = n - q
    if window:
        return sum(min(window, lo + j + 1) for j in range(q)), n - max(0, lo - window + 1)
    return q * lo + q * (q + 1) // 2, n


def work(c):
    lens, Hq, Hkv, d = _lengths(c), c["Hq"], c["Hkv"], c["d"]
    T = sum(q for q, _ in lens)
    four = d // 2 + d // 16  # bytes of a key or a value in 4 bits: codes and scales
    if c["op"] == "append4":  # keys and values in; codes, scales and the values that they stand for out
        table = sum((kv - 1) // c["page"] - (kv - q) // c["page"] + 1 for q, kv in lens)
        return {"bytes": 2 * T * Hkv * (4 * d + four) + 4 * (table + 2 * c["S"]), "flops": 4 * T * Hkv * d}
    if c["op"] == "evict":  # all weights in; kept keys, values and weights in and out, and their places
        n, new = sum(kv for _, kv in lens), sum(min(kv, c["keep"]) for _, kv in lens)
        return {"bytes": Hkv * (4 * n + new * (2 * 4 * d + 8)), "flops": Hkv * n}
    flops = keys = table = 0
    for q, kv in lens:
        p, k = _pairs(q, kv, c["window"])
        flops += (4 if c["op"] == "attn4" else 2) * d * Hq * p
        keys += k
        table += (k + c["page"] - 1) // c["page"]
    if c["op"] == "attn4":
        return {"bytes": 2 * four * Hkv * keys + T * Hq * (4 * d + 4) + 4 * (table + 2 * c["S"]), "flops": flops}
    one = four if c["bits"] == 4 else 2 * d
    return {"bytes": (one + 8) * Hkv * keys + T * Hq * (2 * d + 4) + 4 * (table + 2 * c["S"]), "flops": flops}


def _cost(c):
    w = work(c)
    return w["bytes"] / HBM + w["flops"] / MMA


# --------------------------------------------------------------------------------------------------------- inputs
def _pack(codes):
    """Codes [..., d] as bytes [..., d / 2]."""
    u = codes.to(torch.uint8).unflatten(-1, (-1, 4, 2)).transpose(-1, -2).unflatten(-1, (2, 2))  # [..., d / 8, e, j / 2, j % 2]
    return (u[..., 0] | u[..., 1] << 4).flatten(-3)


def _unpack(x):
    """Bytes [..., d / 2] as codes [..., d], fp32."""
    u = torch.stack([x & 15, x >> 4], -1).unflatten(-2, (-1, 2, 2)).flatten(-2)  # [..., d / 8, e, j]
    return u.transpose(-1, -2).flatten(-3).float()


def _values(codes, scales):
    """What codes [..., d / 2] and scales [..., d / 32] stand for, fp32 [..., d]."""
    return ((_unpack(codes) - 8).unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _quantise(x):
    """(codes 1..15 [..., d], scales [..., d / 32] bf16) of x [..., d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    m, e = torch.frexp(top / torch.full_like(top, 7))  # (a quotient: the product with 1 / 7 misses ties)
    scale = torch.ldexp(torch.round(m * 16) / 16, e).to(torch.bfloat16)  # (the power may be off by an fp32 step)
    one = torch.where(scale > 0, scale, torch.ones_like(scale)).float()
    return (torch.round(g / one[..., None]) + 8).flatten(-2), scale


def _data(c, seed):
    """The tensors of a case, from its seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    Hq, Hkv, d, S, page, op = c["Hq"], c["Hkv"], c["d"], c["S"], c["page"], c["op"]
    lens = _lengths(c)
    pages = [(kv + page - 1) // page for _, kv in lens]
    to = [(min(kv, c["keep"]) + page - 1) // page for _, kv in lens] if op == "evict" else []
    num_pages = sum(pages) + sum(to) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32).cpu()

    def table(counts, at):
        t = torch.zeros(S, max(counts), dtype=torch.int32)
        for i, n in enumerate(counts):
            t[i, :n] = order[at:at + n]
            at += n
        return t.cuda()

    cu = [0]
    for q, _ in lens:
        cu.append(cu[-1] + q)
    T = cu[-1]
    s = {"T": T, "table": table(pages, 0), "cu_q": torch.tensor(cu, dtype=torch.int32).cuda(),
         "kv_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32).cuda()}
    if op == "append4" or c.get("bits") == 4 or op == "attn4":
        for x in "kv":
            codes, scale = _quantise(normal(num_pages, Hkv, page, d))
            s[x + "_codes"], s[x + "_scale"] = _pack(codes), scale
    else:
        s["k_cache"] = normal(num_pages, Hkv, page, d)
    if op == "append4":
        qkv = normal(T, Hq + 2 * Hkv, d)  # a fused projection's output, keys turned in place; k and v are views of it
        s["k"], s["v"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["k_out"], s["v_out"] = (torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "evict":
        s["v_cache"] = normal(num_pages, Hkv, page, d)
        s["to"] = table(to, sum(pages))
        s["keep"] = torch.full((S,), c["keep"], dtype=torch.int32, device="cuda")
    else:
        s["q"] = normal(T, Hq, d)
    if op in ("weights", "evict"):  # a few tokens hold most of the weight; what has vanished in fp32 is equal
        w = torch.randn(num_pages, Hkv, page, generator=g, device="cuda")
        s["weights"] = torch.where(w > -2, torch.exp(3 * w), torch.zeros_like(w))
    if op == "weights":
        s["out"] = s["weights"].clone()
        seen = s["kv_lens"].repeat_interleave(s["cu_q"].diff().long()).float()
        if c["window"]:
            seen = seen.clamp(max=c["window"])
        s["lse"] = (torch.log(seen) + 0.5)[:, None] + 0.2 * torch.randn(T, Hq, generator=g, device="cuda")
    return s


def prepare(case, seed):
    s = _data(case, seed)
    s["case"] = case
    if own:
        from online_softmax_09_gb300 import fa

        if "k_codes" in s:
            s["cache"] = fa.PagedCache4(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        # A serving step's plan, which all its layers share.
        s["plan"] = fa.paged_plan(s["cu_q"], s["kv_lens"], s["table"], num_tokens=s["T"], max_q=max(q for q, _ in _lengths(case)),
                                  page_size=case["page"], Hq=case["Hq"], Hkv=case["Hkv"], d=case["d"], causal=True,
                                  window=case.get("window", 0))
    return s


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from online_softmax_09_gb300 import fa

        if op == "append4":
            fa.paged_append4(None, s["k"], s["v"], s["cache"], s["plan"], k_out=s["k_out"], v_out=s["v_out"])
            return s["k_out"], s["v_out"]
        if op == "attn4":
            return fa.forward_paged4(s["q"], s["cache"], s["plan"])
        if op == "weights":
            return fa.paged_weights(s["q"], s["lse"], s["cache"] if c["bits"] == 4 else s["k_cache"], s["weights"], s["plan"],
                                    out=s["out"])
        kept, lens = fa.paged_evict(s["weights"], (s["k_cache"], s["v_cache"]), s["plan"], s["keep"], s["to"],
                                    max_keep=c["keep"], sinks=c["sinks"], recent=c["recent"])
        return kept, lens, s["k_cache"], s["v_cache"], s["weights"]
    return {"append4": _plain_append, "attn4": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _plain_append(s):
    page = s["case"]["page"]
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)  # the sequence of each token
    pos = s["kv_lens"][seq] - s["cu_q"][seq + 1] + t
    where, slot = s["table"][seq, pos // page].long(), pos % page
    for x in "kv":
        codes, scale = _quantise(s[x])
        s[x + "_codes"][where, :, slot] = _pack(codes)
        s[x + "_scale"][where, :, slot] = scale
        s[x + "_out"].copy_(((codes - 8).unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2))
    return s["k_out"], s["v_out"]


def _gather(s, x):
    """x [pages, Hkv, page, ...] of every sequence's cached tokens, filled up to the longest: [S, Hkv, n, ...]."""
    return x[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :max(kv for _, kv in _lengths(s["case"]))]


def _scores(s, k):
    """Scores [S, Hkv, G, q, n] of the step's tokens, -inf where they see nothing, and the rows of the tokens [S, q]."""
    c = s["case"]
    Hkv, G, n = c["Hkv"], c["Hq"] // c["Hkv"], k.shape[2]
    ql = s["cu_q"].diff()
    j = torch.arange(max(q for q, _ in _lengths(c)), device="cuda")
    row = (s["cu_q"][:-1, None] + j).clamp(max=s["T"] - 1)
    q = s["q"][row].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (G, -1)) / math.sqrt(c["d"])
    pos = (s["kv_lens"] - ql)[:, None] + j
    key = torch.arange(n, device="cuda")
    hide = (key > pos[..., None]) | (j >= ql[:, None])[..., None]
    if c["window"]:
        hide = hide | (key <= pos[..., None] - c["window"])
    return x.masked_fill_(hide[:, None, None], -math.inf), row, j < ql[:, None]


def _plain_attn(s):
    c = s["case"]
    k = _values(_gather(s, s["k_codes"]), _gather(s, s["k_scale"]))
    v = _values(_gather(s, s["v_codes"]), _gather(s, s["v_scale"]))
    x, row, new = _scores(s, k)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)  # (rows that only fill up see nothing)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, x.shape[2:4]) / total
    out = torch.empty(s["T"], c["Hq"], c["d"], dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["T"], c["Hq"], dtype=torch.float32, device="cuda")
    out[row[new]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[new].to(torch.bfloat16)
    lse[row[new]] = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[new]
    return out, lse


def _plain_weights(s):
    c = s["case"]
    page = c["page"]
    k = _values(_gather(s, s["k_codes"]), _gather(s, s["k_scale"])) if c["bits"] == 4 else _gather(s, s["k_cache"]).float()
    x, row, _ = _scores(s, k)
    lse = s["lse"][row].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1)
    w = x.sub_(lse[..., None]).exp_().sum((2, 3))  # [S, Hkv, n]
    n = torch.arange(w.shape[2], device="cuda")
    first = s["kv_lens"] - s["cu_q"].diff()  # tokens from here on are new: nothing has been added up for them
    seen = n < s["kv_lens"][:, None]
    if c["window"]:
        seen = seen & (n > (first - c["window"])[:, None])
    w = w + torch.where(n < first[:, None], 1.0, 0.0)[:, None] * _gather(s, s["weights"])
    i, t = seen.nonzero(as_tuple=True)
    s["out"][s["table"][i, t // page].long(), :, t % page] = w.transpose(1, 2)[i, t]
    return s["out"]


def _plain_evict(s):
    c = s["case"]
    page, keep = c["page"], c["keep"]
    w = _gather(s, s["weights"])
    kv = s["kv_lens"][:, None, None]
    new = torch.minimum(kv, s["keep"][:, None, None])
    sinks = new.clamp(max=c["sinks"])
    recent = torch.minimum(new - sinks, torch.full_like(new, c["recent"]))
    n = torch.arange(w.shape[2], device="cuda")
    w = w.masked_fill(((n < sinks) | (n >= kv - recent)), math.inf).masked_fill(n >= kv, -1)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices  # (equal weights: the lowest place first)
    gone = torch.ones_like(w, dtype=torch.bool).scatter_(2, best, (n >= new).expand_as(w))
    kept = torch.sort(gone.to(torch.uint8), dim=-1, stable=True).indices[..., :keep].int()
    at = torch.arange(kept.shape[2], device="cuda")
    kept = kept.masked_fill(at >= new, -1)
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[2]), value=-1)
    i, h, a = (kept >= 0).nonzero(as_tuple=True)
    src, dst = (s["table"][i, kept[i, h, a] // page].long(), h, kept[i, h, a] % page), (s["to"][i, a // page].long(), h, a % page)
    for x in ("k_cache", "v_cache", "weights"):
        s[x][dst] = s[x][src]
    return kept, new[:, 0, 0], s["k_cache"], s["v_cache"], s["weights"]


# ---------------------------------------------------------------------------------------------------------- exact
def _exact_values(codes, scales):
    """Word by word: [..., d / 2] bytes and their scales as 64-bit values."""
    word = codes.contiguous().view(torch.int32).long() & 0xFFFFFFFF
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    for i in range(8):
        out[..., i::8] = ((word >> (4 * (i // 2) + 16 * (i % 2))) % 16 - 8).double()
    return out * scales.double().repeat_interleave(GROUP, -1)


def _exact_quantised(x):
    """The nearest representable values of x [..., d], group by group, in 64 bits."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    q = top / torch.full_like(top, 7)
    unit = (q.view(torch.int64) >> 52 << 52).view(torch.float64) / 8  # of four significant bits
    scale = torch.where(q > 0, torch.round(q / unit) * unit, q)
    return torch.where(scale > 0, torch.round(g / scale) * scale, torch.zeros_like(g)).flatten(-2)


def exact(case, seed):
    c = case
    lens, Hkv, d, page = _lengths(c), c["Hkv"], c["d"], c["page"]
    if c["op"] in ("attn4", "weights") and work(dict(c, window=0))["flops"] > 8e12:  # about 20 seconds at the 64-bit rate
        return None
    s = _data(c, seed)
    if c["op"] == "append4":
        return _exact_quantised(s["k"]), _exact_quantised(s["v"])
    if c["op"] == "evict":
        return _exact_evict(s, c)
    G, T = c["Hq"] // Hkv, s["T"]
    o = torch.zeros(T, c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, c["Hq"], dtype=torch.float64, device="cuda")
    out = s["out"].double() if c["op"] == "weights" else None
    at = 0
    for i, (ql, n) in enumerate(lens):
        ids = s["table"][i, :(n + page - 1) // page].long()
        here = torch.arange(n, device="cuda")

        def head(x, h):
            return x[:, h][ids].flatten(0, 1)[:n]

        for h in range(Hkv):
            if "k_codes" in s:
                K = _exact_values(head(s["k_codes"], h), head(s["k_scale"], h))
            else:
                K = head(s["k_cache"], h).double()
            V = _exact_values(head(s["v_codes"], h), head(s["v_scale"], h)) if c["op"] == "attn4" else None
            sums = torch.zeros(n, dtype=torch.float64, device="cuda")
            for hq in range(h * G, (h + 1) * G):
                x = s["q"][at:at + ql, hq].double() @ K.T * d ** -0.5
                p = here[n - ql:, None]
                seen = here <= p
                if c["window"]:
                    seen &= here > p - c["window"]
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                if c["op"] == "attn4":
                    z = torch.logsumexp(x, -1)
                    o[at:at + ql, hq] = torch.exp(x - z[:, None]) @ V
                    lse[at:at + ql, hq] = z
                else:
                    sums += torch.exp(x - s["lse"][at:at + ql, hq, None].double()).sum(0)
            if c["op"] == "weights":
                lo = max(0, n - ql - c["window"] + 1) if c["window"] else 0
                old = head(s["weights"], h).double()
                old[n - ql:] = 0
                t = here[lo:]
                out[ids[t // page], h, t % page] = (old + sums)[lo:]
        at += ql
    return out if c["op"] == "weights" else (o, lse)


def _exact_evict(s, c):
    """One sequence and head at a time: the weights above a bound, and the first of those at it."""
    page, keep = c["page"], c["keep"]
    kept = torch.full((c["S"], c["Hkv"], keep), -1, dtype=torch.int32, device="cuda")
    out = {x: s[x].double() for x in ("k_cache", "v_cache", "weights")}
    new_lens = []
    for i, (_, n) in enumerate(_lengths(c)):
        new = min(n, keep)
        new_lens.append(new)
        ids, to = s["table"][i].long(), s["to"][i].long()
        a = min(c["sinks"], new)
        b = n - min(c["recent"], new - a)
        m = new - a - (n - b)  # of places a .. b
        for h in range(c["Hkv"]):
            w = s["weights"][:, h][ids].flatten()[a:b].double()
            place = torch.zeros(0, dtype=torch.long, device="cuda")
            if m > 0:
                bound = torch.sort(w).values[w.numel() - m]
                above = w > bound
                level = (w == bound).nonzero()[:, 0][:m - int(above.sum())]
                place = torch.cat([above.nonzero()[:, 0], level]).sort().values + a
            src = torch.cat([torch.arange(a, device="cuda"), place, torch.arange(b, n, device="cuda")])
            dst = torch.arange(new, device="cuda")
            kept[i, h, :new] = src.int()
            for x in out:
                out[x][to[dst // page], h, dst % page] = s[x][ids[src // page], h, src % page].double()
    return kept, torch.tensor(new_lens, dtype=torch.int32, device="cuda"), out["k_cache"], out["v_cache"], out["weights"]
