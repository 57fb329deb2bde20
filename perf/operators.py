"""Cases, plain forms and 64-bit definitions of the rotary, cache-append and paged-attention operators.

Every case is a dict of plain values; ``prepare`` makes what a user's program holds before the call, ``run`` is one pass
(elementary torch operations in fp32 where ``own`` is false, the library's entry points where it is true) and ``exact``
the same outputs in 64 bits.
"""

import math
import random

import torch

own = False

HBM = 6.7e12  # bytes/s and flop/s used only to compare the cost of drawn cases with the listed ones
MMA = 1.9e15


# ---------------------------------------------------------------------------------------------------------- cases
def _rope(name, B, Hq, Hkv, N, d, rot, interleaved, sections, theta, start):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "rot": rot,
            "interleaved": interleaved, "sections": sections, "theta": theta, "start": start}


def _append(name, S, q_min, q_max, kv_min, kv_max, Hq, Hkv, d, page, rot, interleaved, theta, lens):
    return {"name": name, "op": "append", "S": S, "q_min": q_min, "q_max": q_max, "kv_min": kv_min, "kv_max": kv_max,
            "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "rot": rot, "interleaved": interleaved, "theta": theta,
            "lens": lens}


def _attn(name, S, q_min, q_max, kv_min, kv_max, Hq, Hkv, d, page, window, lens, chunk=0):
    return {"name": name, "op": "attn", "S": S, "q_min": q_min, "q_max": q_max, "kv_min": kv_min, "kv_max": kv_max,
            "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "window": window, "lens": lens, "chunk": chunk}


def listed():
    return [
        # A training step's q and k (Llama-3.1-8B heads, the benchmark's shape), read out of the fused projection, rotated
        # for the attention kernels, and the gradients rotated back.
        _rope("rope-train-b4-n4096", 4, 32, 8, 4096, 128, 128, False, "", 5.0e5, 0),
        # Video tokens with (time, height, width) positions, an odd number of them, d = 64.
        _rope("rope-video-3axes-n4111", 2, 16, 16, 4111, 64, 64, False, "8,12,12", 1.0e4, 20000),
        # One short prompt far into a conversation, adjacent pairs, half of the dims rotated: latency.
        _rope("rope-short-n17", 1, 32, 8, 17, 128, 64, True, "", 1.0e4, 120000),
        # One new token of one conversation: latency.
        _append("append-one-token", 1, 1, 1, 1000, 1000, 32, 8, 128, 16, 128, False, 5.0e5, 1),
        # A decode step of 64 conversations.
        _append("append-decode-s64", 64, 1, 1, 100, 2000, 32, 8, 128, 16, 128, False, 5.0e5, 2),
        # Prompts of ragged lengths brought into the cache together.
        _append("append-prompts-s8", 8, 300, 1900, 1900, 2500, 32, 8, 128, 64, 128, False, 5.0e5, 3),
        # One new token of one conversation of about a thousand tokens: latency.
        _attn("attn-one-token-kv1000", 1, 1, 1, 1000, 1000, 32, 8, 128, 16, 0, 4),
        # A decode step of 64 conversations of ragged lengths.
        _attn("attn-decode-s64", 64, 1, 1, 200, 8192, 32, 8, 128, 16, 0, 5),
        # Four drafted tokens checked for each of 48 conversations, d = 64, a sliding window.
        _attn("attn-draft4-s48-window", 48, 4, 4, 500, 6000, 16, 4, 64, 32, 1024, 6),
        # Two conversations as long as the long-context benchmark, one token each.
        _attn("attn-long-s2-kv131072", 2, 1, 1, 120001, 131072, 32, 8, 128, 64, 0, 7),
        # The next chunk of one long prompt.
        _attn("attn-chunk512-kv32768", 1, 512, 512, 32768, 32768, 32, 8, 128, 64, 0, 8),
        # A serving step that mixes single tokens with one prompt's chunk of an odd length.
        _attn("attn-mixed-s24", 24, 1, 1, 300, 9000, 32, 8, 128, 16, 0, 9, 4097),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: each operator alike often, sizes log-uniform over the listed range, at most the largest listed cost."""
    cap = max(_cost(c) for c in listed())
    op = rng.choice(["rope", "append", "attn"])
    while True:
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 5, 8, 16])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        if op == "rope":
            sections = rng.choice(["", "", "3"])
            rot = rng.choice([d, d, d // 2])
            if sections:
                a = rng.randint(1, rot // 2 - 2)
                b = rng.randint(1, rot // 2 - a - 1)
                sections = "%d,%d,%d" % (a, b, rot // 2 - a - b)
            c = _rope(None, _log(rng, 1, 8), Hkv * G, Hkv, _log(rng, 1, 16384), d, rot, rng.random() < 0.3, sections,
                      rng.choice([1.0e4, 5.0e5]), rng.choice([0, _log(rng, 1, 120000)]))
        elif op == "append":
            q_max = rng.choice([1, 1, _log(rng, 2, 4096)])
            kv_max = q_max + _log(rng, 1, 4096)
            c = _append(None, _log(rng, 1, 128), rng.choice([1, q_max]), q_max, q_max, kv_max, Hkv * G, Hkv, d,
                        rng.choice([16, 32, 64, 128]), rng.choice([d, d, d // 2]), rng.random() < 0.3,
                        rng.choice([1.0e4, 5.0e5]), rng.randint(0, 10 ** 6))
            if sum(n for _, n in _lengths(c)) * Hkv * d > 2 ** 28:  # the whole cache is an output
                continue
        else:
            q_max = rng.choice([1, 1, _log(rng, 2, 4096)])
            kv_max = max(q_max, _log(rng, 16, 131072))
            kv_min = max(q_max, _log(rng, 1, kv_max))
            window = rng.choice([0, 0, _log(rng, 16, 8192)])
            c = _attn(None, _log(rng, 1, 128), rng.choice([1, q_max]), q_max, kv_min, kv_max, Hkv * G, Hkv, d,
                      rng.choice([16, 32, 64, 128]), window, rng.randint(0, 10 ** 6))
            if sum(n for _, n in _lengths(c)) * Hkv * d > 2 ** 31:
                continue
        if _cost(c) <= cap:
            del c["name"]
            return c


def _lengths(c):
    """(new tokens, cached tokens with them) of every sequence; the case alone decides."""
    r = random.Random(c["lens"])
    out = [(r.randint(c["q_min"], c["q_max"]), r.randint(c["kv_min"], c["kv_max"])) for _ in range(c["S"])]
    if c.get("chunk"):  # one prompt's chunk among single tokens
        i = r.randrange(c["S"])
        out[i] = (c["chunk"], 2 * c["chunk"] + 11)
    return out


def _pairs(q, n, window):
    """Visible (query token, key) pairs and the number of keys that any of the q last queries of n positions sees."""
    lo = n - q
    total = 0
    if window:
        total = sum(min(window, lo + j + 1) for j in range(q))
        return total, n - max(0, lo - window + 1)
    return q * lo + q * (q + 1) // 2, n


def work(c):
    if c["op"] == "rope":  # forward of q and k, backward of their gradients
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        A = len(c["sections"].split(",")) if c["sections"] else 1
        return {"bytes": 8 * n + 4 * A * c["N"] + 2 * c["rot"], "flops": 6 * n}
    lens = _lengths(c)
    T = sum(q for q, _ in lens)
    if c["op"] == "append":
        n = T * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        table = sum((kv - 1) // c["page"] - (kv - q) // c["page"] + 1 for q, kv in lens)
        return {"bytes": 4 * n + 4 * (table + 2 * c["S"]) + 2 * c["rot"], "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    d, flops, keys, table = c["d"], 0, 0, 0
    for q, kv in lens:
        p, k = _pairs(q, kv, c["window"])
        flops += 4 * d * c["Hq"] * p
        keys += k
        table += (k + c["page"] - 1) // c["page"]
    return {"bytes": 4 * d * c["Hkv"] * keys + T * c["Hq"] * (4 * d + 4) + 4 * (table + 2 * c["S"]), "flops": flops}


def _cost(c):
    w = work(c)
    return w["bytes"] / HBM + w["flops"] / MMA


# --------------------------------------------------------------------------------------------------------- inputs
def _inv_freq(c):
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
    return (c["theta"] ** (-i / c["rot"])).to(torch.float32).cuda()


def _axes(c):
    """The axis of each rotated pair, or None for one axis."""
    if not c.get("sections"):
        return None
    return [a for a, n in enumerate(c["sections"].split(",")) for _ in range(int(n))]


def _positions(c, g):
    """[N] for one axis; (time, height, width) of frames of 16 x 24 patches after some text for three."""
    n = torch.arange(c["N"], dtype=torch.int32)
    if not c["sections"]:
        return (n + c["start"]).cuda()
    return torch.stack([n // 384 + c["start"], n // 24 % 16 + c["start"], n % 24 + c["start"]]).to(torch.int32).cuda()


def _data(c, seed):
    """The tensors of a case, from its seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    s = {}
    if c["op"] == "rope":
        B, N = c["B"], c["N"]
        qkv = normal(B, N, Hq + 2 * Hkv, d)  # a fused projection's output; q and k are views of it
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["dq"] = normal(B, Hq, N, d)  # gradients as the attention backward writes them
        s["dk"] = normal(B, Hkv, N, d)
        s["positions"] = _positions(c, g)
        s["inv_freq"] = _inv_freq(c)
        return s
    lens = _lengths(c)
    S, page = c["S"], c["page"]
    pages = [(kv + page - 1) // page for _, kv in lens]
    num_pages = sum(pages) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(S, max(pages), dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    cu = [0]
    for q, _ in lens:
        cu.append(cu[-1] + q)
    T = cu[-1]
    s["lens"] = lens
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32).cuda()
    s["kv_lens"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32).cuda()
    s["table"] = table.cuda()
    s["k_cache"] = normal(num_pages, Hkv, page, d)
    s["v_cache"] = normal(num_pages, Hkv, page, d)
    if c["op"] == "append":
        qkv = normal(T, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["inv_freq"] = _inv_freq(c)
    else:
        s["q"] = normal(T, Hq, d)
    return s


def prepare(case, seed):
    s = _data(case, seed)
    s["case"] = case
    if own:
        from online_softmax_09_gb300 import fa

        if "inv_freq" in s:
            s["rotary"] = fa.Rotary(s["inv_freq"], interleaved=case["interleaved"], axes=_axes(case))
        if case["op"] != "rope":  # a serving step's plan, which all its layers share
            s["plan"] = fa.paged_plan(s["cu_q"], s["kv_lens"], s["table"], num_tokens=s["q"].shape[0],
                                      max_q=max(q for q, _ in s["lens"]), page_size=case["page"], Hq=case["Hq"],
                                      Hkv=case["Hkv"], d=case["d"], causal=True, window=case.get("window", 0))
    return s


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    op = s["case"]["op"]
    if own:
        from online_softmax_09_gb300 import fa

        if op == "rope":
            q, k = fa.rope(s["q"], s["k"], s["positions"], s["rotary"])
            dq, dk = fa.rope_backward(s["dq"], s["dk"], s["positions"], s["rotary"])
            return q, k, dq, dk
        if op == "append":
            q = fa.paged_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["plan"], s["rotary"])
            return q, s["k_cache"], s["v_cache"]
        return fa.forward_paged(s["q"], s["k_cache"], s["v_cache"], s["plan"])
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](s)


def _turn(x, cos, sin, rot, interleaved):
    """x [..., d] rotated in fp32 by the angles whose cos and sin [..., rot / 2] are given, rounded once."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _cos_sin(c, positions, inv_freq):
    """cos and sin of position * frequency, the angle in 64 bits: [N, rot / 2]."""
    axes = _axes(c)
    pos = positions.double()
    pos = pos[torch.tensor(axes, device=pos.device)].T if axes else pos[:, None]
    phi = pos * inv_freq.double()
    return phi.cos().float(), phi.sin().float()


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(c, s["positions"], s["inv_freq"])
    a = (c["rot"], c["interleaved"])
    return (_turn(s["q"], cos, sin, *a).contiguous(), _turn(s["k"], cos, sin, *a).contiguous(),
            _turn(s["dq"], cos, -sin, *a), _turn(s["dk"], cos, -sin, *a))


def _plain_append(s):
    c = s["case"]
    page = c["page"]
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = (t[:, None] >= s["cu_q"][None, 1:]).sum(1)  # the sequence of each token
    pos = s["kv_lens"][seq] - s["cu_q"][seq + 1] + t
    cos, sin = _cos_sin({"sections": ""}, pos, s["inv_freq"])
    cos, sin = cos[:, None], sin[:, None]
    q = _turn(s["q"], cos, sin, c["rot"], c["interleaved"])
    k = _turn(s["k"], cos, sin, c["rot"], c["interleaved"])
    where = s["table"][seq, pos // page].long()
    s["k_cache"][where, :, pos % page] = k
    s["v_cache"][where, :, pos % page] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, d, page, window = c["Hq"], c["Hkv"], c["d"], c["page"], c["window"]
    G = Hq // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    at = 0
    for i, (ql, n) in enumerate(s["lens"]):
        first = max(0, n - ql - window + 1) // page if window else 0  # the first page that a query sees
        ids = s["table"][i, first:(n + page - 1) // page].long()
        k = s["k_cache"][ids].transpose(0, 1).reshape(Hkv, -1, d).float()
        v = s["v_cache"][ids].transpose(0, 1).reshape(Hkv, -1, d).float()
        key = torch.arange(k.shape[1], device="cuda") + first * page
        step = max(1, 2 ** 29 // (Hq * k.shape[1]))
        for j in range(0, ql, step):
            m = min(step, ql - j)
            q = s["q"][at + j:at + j + m].float().view(m, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * m, d)
            x = torch.matmul(q, k.transpose(1, 2)).view(Hkv, G, m, -1) / math.sqrt(d)
            p = torch.arange(j, j + m, device="cuda")[:, None] + (n - ql)
            hide = key[None] > p
            if window:
                hide = hide | (key[None] <= p - window)
            x = x.masked_fill(hide, -math.inf)
            top = x.amax(-1, keepdim=True)
            x = torch.exp(x - top)
            total = x.sum(-1, keepdim=True)
            o = torch.matmul(x.view(Hkv, G * m, -1), v).view(Hkv, G, m, d) / total
            out[at + j:at + j + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, d).to(torch.bfloat16)
            lse[at + j:at + j + m] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(m, Hq)
        at += ql
    return out, lse


# ---------------------------------------------------------------------------------------------------------- exact
def _exact_turn(x, pos, inv_freq, rot, interleaved, sign):
    """The rotation as a product with unit complex numbers in 64 bits; pos [..., rot / 2] is each pair's position."""
    x = x.double()
    phase = sign * pos.double() * inv_freq.double()
    unit = torch.polar(torch.ones_like(phase), phase)
    if interleaved:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * unit
        r = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * unit
        r = torch.cat([z.real, z.imag], -1)
    return torch.cat([r, x[..., rot:]], -1)


def exact(case, seed):
    c = case
    if c["op"] == "attn" and work(dict(c, window=0))["flops"] > 8e12:  # about 20 seconds at this card's 64-bit rate
        return None
    s = _data(c, seed)
    if c["op"] == "rope":
        axes = _axes(c) or [0] * (c["rot"] // 2)
        table = s["positions"].reshape(-1, c["N"])
        pos = torch.stack([table[a] for a in axes], -1)
        return tuple(_exact_turn(s[n], pos, s["inv_freq"], c["rot"], c["interleaved"], sign)
                     for n, sign in (("q", 1), ("k", 1), ("dq", -1), ("dk", -1)))
    if c["op"] == "append":
        kc, vc, q_out = s["k_cache"].double(), s["v_cache"].double(), []
        at = 0
        for i, (ql, n) in enumerate(s["lens"]):
            pos = torch.arange(n - ql, n, device="cuda")
            turned = [_exact_turn(s[t][at:at + ql], pos[:, None, None], s["inv_freq"], c["rot"], c["interleaved"], 1)
                      for t in ("q", "k")]
            q_out.append(turned[0])
            for b in range((n - ql) // c["page"], (n - 1) // c["page"] + 1):  # page by page
                lo, hi = max(b * c["page"], n - ql), min((b + 1) * c["page"], n)
                src, dst = slice(lo - n + ql, hi - n + ql), slice(lo - b * c["page"], hi - b * c["page"])
                pid = int(s["table"][i, b])
                kc[pid, :, dst] = turned[1][src].transpose(0, 1)
                vc[pid, :, dst] = s["v"][at:at + ql][src].double().transpose(0, 1)
            at += ql
        return torch.cat(q_out), kc, vc
    return _exact_attn(s, c)


def _exact_attn(s, c):
    """One head of queries at a time, its scores in 64 bits, keys of one sequence in one piece."""
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for i, (ql, n) in enumerate(s["lens"]):
        row = s["table"][i, :(n + page - 1) // page].long()
        here = torch.arange(n, device="cuda")
        for h in range(Hkv):
            K = s["k_cache"][:, h][row].reshape(-1, d)[:n].double()
            V = s["v_cache"][:, h][row].reshape(-1, d)[:n].double()
            step = max(1, 2 ** 27 // n)
            heads = range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for j in range(0, ql, step):
                p = here[n - ql:][j:j + step, None]
                seen = here <= p
                if c["window"]:
                    seen &= here > p - c["window"]
                for hq in heads:
                    x = s["q"][at + j:at + min(j + step, ql), hq].double() @ K.T * d ** -0.5
                    x = torch.where(seen, x, torch.full_like(x, -math.inf))
                    z = torch.logsumexp(x, -1)
                    o[at + j:at + min(j + step, ql), hq] = torch.exp(x - z[:, None]) @ V
                    lse[at + j:at + min(j + step, ql), hq] = z
        at += ql
    return o, lse
