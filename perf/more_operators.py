"""Cases of the dense-attention side of a layer, in a plain torch form and as calls of this library.

    table  cos / sin table of rotary positions, plain or scaled for long contexts             (dsa_rope_table)
    rope   rotation of heads by such a table, either pair layout, any part of the head        (dsa_rope)
    qk     per-head RMS norm + rotation of queries and keys, keys and values to a paged cache  (dsa_qk_norm_rope)
    attn   attention of new tokens over a paged bf16 cache                                     (dsa_paged_attn)

A layer that attends to every cached key (a draft layer, a layer without the selection, a prompt no longer than the
selection) runs them in this order: the table is made once, the projected heads are normalised and rotated while keys
and values go to their cache slots, the attention reads the cache, and the rotation of its output is taken back where
values carry positions.

`own` chooses between the plain form (False) and the library's calls (True).
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


_calls = None


def _lib():
    global _calls
    if _calls is None:
        from deepseek_v4_sparse_dsa_gb300 import dsa
        _calls = dsa
    return _calls


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the table of a short context, made when a model is loaded
        {"name": "table 4096x64", "op": "table", "n": 4096, "R": 64, "pos0": 0, "scaling": "plain", "factor": 1.0},
        # a million positions, sixteen times what the frequencies were trained for
        {"name": "table 1M x 64 yarn", "op": "table", "n": 1 << 20, "R": 64, "pos0": 0, "scaling": "yarn", "factor": 16.0},
        # a decode batch's attention output, whose last 64 of 128 dims are turned back
        {"name": "rope 64x64x128 inverse", "op": "rope", "T": 64, "H": 64, "D": 128, "R": 64, "off": 64, "pad": 0,
         "layout": "interleaved", "inverse": True, "type": "bf16"},
        # the queries of a chunk of 8192 tokens, all dims, halves rotated against each other
        {"name": "rope 8192x64x128 half", "op": "rope", "T": 8192, "H": 64, "D": 128, "R": 128, "off": 0, "pad": 0,
         "layout": "half", "inverse": False, "type": "bf16"},
        # one token: nothing but latency
        {"name": "qk 1x64+8x128", "op": "qk", "T": 1, "H": 64, "Hkv": 8, "D": 128, "R": 128, "off": 0, "layout": "half",
         "norm": True, "type": "bf16", "bs": 64},
        # an odd batch of an odd number of fp32 heads, of which only a part turns
        {"name": "qk 517x7+1x80 f32", "op": "qk", "T": 517, "H": 7, "Hkv": 1, "D": 80, "R": 40, "off": 40,
         "layout": "interleaved", "norm": True, "type": "f32", "bs": 20},
        # a chunk of 8192 tokens
        {"name": "qk 8192x64+8x128", "op": "qk", "T": 8192, "H": 64, "Hkv": 8, "D": 128, "R": 64, "off": 64,
         "layout": "interleaved", "norm": True, "type": "bf16", "bs": 64},
        # one token of one sequence over 4096 cached ones: latency, and the split of one row over the GPU
        {"name": "attn 1x1 ctx 4096", "op": "attn", "B": 1, "each": 1, "tokens": 1, "ctx": 4096, "H": 64, "Hkv": 8, "D": 128,
         "bs": 64, "window": 0, "sink": False},
        # a decode batch over contexts up to 32K: bound by the cache's stream from memory
        {"name": "attn 64x1 ctx 32768", "op": "attn", "B": 64, "each": 1, "tokens": 64, "ctx": 32768, "H": 64, "Hkv": 8,
         "D": 128, "bs": 64, "window": 0, "sink": False},
        # two tokens per sequence (one drafted) of 64 heads that share one key head, a window and sinks
        {"name": "attn 32x2 window 4096", "op": "attn", "B": 32, "each": 2, "tokens": 64, "ctx": 131072, "H": 64, "Hkv": 1,
         "D": 128, "bs": 64, "window": 4096, "sink": True},
        # a mixed step: 12 requests bring 2000 tokens unevenly to contexts up to 5000, six query heads per key head
        {"name": "attn 12 mixed", "op": "attn", "B": 12, "each": 0, "tokens": 2000, "ctx": 5000, "H": 24, "Hkv": 4, "D": 64,
         "bs": 16, "window": 0, "sink": False},
        # a prompt of 8192 tokens: bound by the tensor cores
        {"name": "attn prompt 8192", "op": "attn", "B": 1, "each": 8192, "tokens": 8192, "ctx": 0, "H": 64, "Hkv": 8, "D": 128,
         "bs": 64, "window": 0, "sink": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "qk", "qk", "attn", "attn", "attn"])
    if op == "table":
        R = 2 * _log(rng, 4, 128)
        return {"op": op, "n": _log(rng, 256, min(1 << 20, (1 << 26) // R)), "R": R,
                "pos0": rng.choice([0, 0, 1, 4096, 1000003]), "scaling": rng.choice(["plain", "linear", "yarn"]),
                "factor": rng.choice([1.0, 2.0, 4.0, 16.0, 40.0])}
    if op in ("rope", "qk"):
        D = rng.choice([8 * _log(rng, 1, 32), 64, 128, 128, 192, 256, 2 * _log(rng, 8, 128)])
        R = min(D, rng.choice([D, D // 2 // 8 * 8, 64, 2 * rng.randint(1, D // 2)]))
        R = max(2, R)
        case = {"op": op, "T": 0, "H": rng.choice([1, 8, 16, 64, rng.randint(1, 64)]), "D": D, "R": R,
                "off": rng.choice([0, D - R, 0, D - R, rng.randint(0, D - R)]), "layout": rng.choice(["interleaved", "half"]),
                "type": rng.choice(["bf16", "bf16", "f32"])}
        if op == "qk":
            case["Hkv"] = rng.choice([h for h in (1, 2, 4, 8, 64) if case["H"] % h == 0])
            case["norm"] = rng.random() < 0.8
            case["bs"] = rng.choice([1, 16, 20, 64, 64, 256])
        else:
            case["pad"] = rng.choice([0, 0, 3, 8])
            case["inverse"] = rng.random() < 0.4
        width = (case["H"] + 2 * case.get("Hkv", 0)) * D * (2 if case["type"] == "f32" else 1)
        case["T"] = _log(rng, 1, max(1, min(16384, 8192 * 64 * 128 // width)))
        return case
    Hkv = rng.choice([1, 1, 2, 4, 8])
    H = Hkv * rng.choice([1, 4, 6, 8, 16, 64 // Hkv])
    D = rng.choice([64, 128, 128])
    B = _log(rng, 1, 128)
    each = rng.choice([0, 0, 1, 1, 2, 4])
    tokens = B * each if each else _log(rng, B, max(B, 4096))
    most = each or tokens                     # what one sequence may bring
    # the cost of the largest listed cases bounds the scores and the cache
    ctx = _log(rng, 1, max(1, min(131072, (1 << 32) // (B * H * most), (1 << 30) // (B * Hkv * D))))
    return {"op": op, "B": B, "each": each, "tokens": tokens, "ctx": ctx, "H": H, "Hkv": Hkv, "D": D,
            "bs": rng.choice([8, 16, 16, 20, 32, 64, 64, 128, 256]), "window": rng.choice([0, 0, 0, 100, 128, 4096]),
            "sink": rng.random() < 0.4}


def _lengths(case):
    """New and cached tokens of each sequence of an attention case: contexts evenly spread up to `ctx`, new tokens the
    same for all or most of them in a few sequences (the ones with short contexts)."""
    B = case["B"]
    cached = [case["ctx"] * (k + 1) // B for k in range(B)]
    if case["each"]:
        return [case["each"]] * B, [max(0, c - case["each"]) for c in cached]
    weight = [((B - k - 0.5) / B) ** 3 for k in range(B)]
    new = [int(w / sum(weight) * case["tokens"]) for w in weight]
    new[0] += case["tokens"] - sum(new)
    return new, cached


# ------------------------------------------------------------------------------------------------ inputs

def _cos_sin(n, R):
    """cos and sin of positions 0 .. n - 1 at the frequencies 10000^(-2i/R)."""
    f = torch.pow(10000.0, -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    s = dict(case)
    if case["op"] == "table":
        # the base varies from model to model, and with it the trained context
        s["base"] = 10000.0 * (1.0 + float(torch.rand((), generator=g, device=dev)))
        s["orig"] = 4096.0
        s["out"] = torch.empty(case["n"], case["R"], device=dev)
    elif case["op"] == "rope":
        T, H, D, typ = case["T"], case["H"], case["D"], TYPES[case["type"]]
        s["x"] = torch.zeros(T, H * D + case["pad"], device=dev, dtype=typ)[:, :H * D]
        s["x"].copy_(randn(T, H * D).to(typ))
        s["pos"] = torch.randint(0, 8192, (T,), generator=g, device=dev, dtype=torch.int32)
        s["cs"] = _cos_sin(8192, case["R"])
        s["y"] = torch.empty(T, H, D, device=dev, dtype=typ)
    elif case["op"] == "qk":
        T, H, Hkv, D, bs, typ = case["T"], case["H"], case["Hkv"], case["D"], case["bs"], TYPES[case["type"]]
        # one projection's output: the heads of queries, keys and values side by side
        s["qkv"] = randn(T, (H + 2 * Hkv) * D).mul_(2.0).to(typ)
        s["gq"], s["gk"] = 1.0 + 0.1 * randn(D), 1.0 + 0.1 * randn(D)
        s["pos"] = torch.randint(0, 8192, (T,), generator=g, device=dev, dtype=torch.int32)
        s["cs"] = _cos_sin(8192, case["R"])
        blocks = -(-T // bs) + 2
        s["slot"] = torch.randperm(blocks * bs, generator=g, device=dev)[:T].contiguous()
        s["kc"] = randn(blocks, bs, Hkv, D).bfloat16()
        s["vc"] = randn(blocks, bs, Hkv, D).bfloat16()
        s["q"] = torch.empty(T, H, D, device=dev, dtype=typ)
    else:
        B, H, Hkv, D, bs = (case[k] for k in ("B", "H", "Hkv", "D", "bs"))
        new, cached = _lengths(case)
        order = torch.randperm(B, generator=g, device=dev)
        new = torch.tensor(new, device=dev, dtype=torch.int32)[order]
        s["ctx_len"] = torch.tensor(cached, device=dev, dtype=torch.int32)[order] + new
        s["new"] = new
        s["start"] = torch.nn.functional.pad(torch.cumsum(new, 0, dtype=torch.int32), (1, 0))
        s["T"], s["most"], s["longest"] = int(new.sum()), int(new.max()), int(s["ctx_len"].max())
        pages = (s["ctx_len"] + (bs - 1)) // bs
        used = int(pages.sum())
        pool = torch.randperm(used + 1, generator=g, device=dev, dtype=torch.int32)
        col = torch.arange(-(-s["longest"] // bs), device=dev, dtype=torch.int32)
        first = torch.cumsum(pages, 0, dtype=torch.int32) - pages
        live = col[None, :] < pages[:, None]
        s["table"] = torch.where(live, pool[torch.where(live, first[:, None] + col, 0).long()], -1)
        s["q"] = randn(s["T"], H, D).mul_(2.0).bfloat16()
        make = lambda: torch.empty(used + 1, bs, Hkv, D, device=dev, dtype=torch.bfloat16).normal_(generator=g)  # noqa: E731
        s["kc"], s["vc"] = make(), make()
        s["sinks"] = randn(H) if case["sink"] else None
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(s["T"], H, D, device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.empty(s["T"], H, device=dev)
        s["ws"] = None
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return {"table": _table, "rope": _rope, "qk": _qk, "attn": _attn}[s["op"]](s)


def _table(s):
    R, n = s["R"], s["n"]
    if own:
        dsa = _lib()
        kind = {"plain": dsa.DSA_ROPE_PLAIN, "linear": dsa.DSA_ROPE_LINEAR, "yarn": dsa.DSA_ROPE_YARN}[s["scaling"]]
        params = dsa.make_rope_params(s["base"], kind, s["factor"], s["orig"])
        dsa.dsa_rope_table(params, R, s["pos0"], n, s["out"])
        return s["out"]
    # angles of far positions need 64 bits
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    f = torch.pow(s["base"], -2.0 * i / R)
    if s["scaling"] == "linear":
        f = f / s["factor"]
    elif s["scaling"] == "yarn":
        pair = lambda turns: R * math.log(s["orig"] / (2 * math.pi * turns)) / (2 * math.log(s["base"]))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / s["factor"] * ramp
    a = torch.arange(s["pos0"], s["pos0"] + n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rotate(x, cs, R, off, layout, inverse=False):
    """x [T, H, D] in fp32 with the pairs of dims [off, off + R) turned by cs [T, R]."""
    c, sn = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if inverse:
        sn = -sn
    part = x[..., off:off + R]
    if layout == "interleaved":
        x0, x1 = part[..., 0::2], part[..., 1::2]
        part = torch.stack([x0 * c - x1 * sn, x0 * sn + x1 * c], -1).flatten(-2)
    else:
        x0, x1 = part[..., :R // 2], part[..., R // 2:]
        part = torch.cat([x0 * c - x1 * sn, x0 * sn + x1 * c], -1)
    return torch.cat([x[..., :off], part, x[..., off + R:]], -1)


def _rope(s):
    T, H, D = s["T"], s["H"], s["D"]
    if own:
        dsa = _lib()
        typ = dsa.DSA_REAL_F32 if s["type"] == "f32" else dsa.DSA_REAL_BF16
        layout = dsa.DSA_ROPE_HALF if s["layout"] == "half" else dsa.DSA_ROPE_INTERLEAVED
        dsa.dsa_rope(s["x"], s["x"].stride(0), D, s["pos"], s["cs"], 8192, s["R"], s["off"], layout, s["inverse"], T, H, D,
                     typ, s["y"], H * D, D)
        return s["y"]
    y = _rotate(s["x"].float().view(T, H, D), s["cs"][s["pos"].long()], s["R"], s["off"], s["layout"], s["inverse"])
    return y.to(TYPES[s["type"]])


def _qk(s):
    T, H, Hkv, D = s["T"], s["H"], s["Hkv"], s["D"]
    ld = (H + 2 * Hkv) * D
    if own:
        dsa = _lib()
        typ = dsa.DSA_REAL_F32 if s["type"] == "f32" else dsa.DSA_REAL_BF16
        layout = dsa.DSA_ROPE_HALF if s["layout"] == "half" else dsa.DSA_ROPE_INTERLEAVED
        gq, gk = (s["gq"], s["gk"]) if s["norm"] else (None, None)
        dsa.dsa_qk_norm_rope(s["qkv"], ld, H, s["qkv"][:, H * D:], ld, Hkv, s["qkv"][:, (H + Hkv) * D:], ld, T, D, typ, gq, gk,
                             EPS, s["pos"], s["cs"], 8192, s["R"], s["off"], layout, s["q"], H * D, None, 0,
                             dsa.make_kv_cache(s["kc"], s["vc"]), s["slot"])
        return {"q": s["q"], "k_cache": s["kc"], "v_cache": s["vc"]}
    x = s["qkv"].float().view(T, H + 2 * Hkv, D)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if s["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["gq"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["gk"]
    cs = s["cs"][s["pos"].long()]
    s["kc"].view(-1, Hkv, D)[s["slot"]] = _rotate(k, cs, s["R"], s["off"], s["layout"]).bfloat16()
    s["vc"].view(-1, Hkv, D)[s["slot"]] = v.bfloat16()
    return {"q": _rotate(q, cs, s["R"], s["off"], s["layout"]).to(TYPES[s["type"]]), "k_cache": s["kc"], "v_cache": s["vc"]}


def _attn(s):
    B, H, Hkv, D, bs, T = (s[k] for k in ("B", "H", "Hkv", "D", "bs", "T"))
    if own:
        dsa = _lib()
        if s["ws"] is None:                   # kept with the layer's other buffers
            s["ws"] = torch.empty(dsa.dsa_paged_attn_workspace_bytes(T, B, H, Hkv, D), device="cuda", dtype=torch.uint8)
        dsa.dsa_paged_attn(s["q"], H * D, T, H, Hkv, D, s["start"], s["ctx_len"], B, s["table"], s["table"].shape[1],
                           dsa.make_kv_cache(s["kc"], s["vc"]), s["scale"], True, s["window"], s["sinks"], s["out"], H * D,
                           s["lse"], s["ws"], s["ws"].numel())
        return {"out": s["out"], "lse": s["lse"]}
    G, dev = H // Hkv, s["q"].device
    j = torch.arange(s["longest"], device=dev, dtype=torch.int32)
    row = s["table"][:, (j // bs).long()].clamp(min=0).long() * bs + j % bs
    i = torch.arange(s["most"], device=dev, dtype=torch.int32)
    token = (s["start"][:-1, None] + i).clamp(max=T - 1).long()
    # every sequence padded to the most new tokens and the longest context: [B, Hkv, tokens x heads, keys]
    q = s["q"][token].float().view(B, -1, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    p = q @ s["kc"].view(-1, Hkv, D)[row].float().permute(0, 2, 3, 1)
    p = p.mul_(s["scale"]).view(B, Hkv, -1, G, s["longest"])
    pos = (s["ctx_len"] - s["new"])[:, None, None] + i[None, :, None]
    hidden = (j > pos) | (j >= s["ctx_len"][:, None, None])
    if s["window"]:
        hidden |= j <= pos - s["window"]
    p.masked_fill_(hidden[:, None, :, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    if s["sinks"] is not None:
        sink = s["sinks"].view(Hkv, 1, G, 1)
        m = torch.maximum(m, sink)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - m).exp()
    o = p.view(B, Hkv, -1, s["longest"]) @ s["vc"].view(-1, Hkv, D)[row].float().transpose(1, 2)
    o = o.view(B, Hkv, -1, G, D) / total
    lse = (m + total.log()).squeeze(-1)
    # back to rows of tokens
    t = torch.arange(T, device=dev, dtype=torch.int32)
    b = torch.searchsorted(s["start"][1:], t, right=True)
    i = (t - s["start"][b]).long()
    return {"out": o.transpose(1, 2)[b, i].reshape(T, H, D).bfloat16(), "lse": lse.transpose(1, 2)[b, i].reshape(T, H)}


# ------------------------------------------------------------------------------------------------ floor and exact values

def _visible(case):
    """(keys of the cache that some row sees, pairs of a token and a key that it sees) of an attention case."""
    keys = pairs = 0
    for n, c in zip(*_lengths(case)):
        if not n:
            continue
        w = case["window"] or c + n
        keys += c + n - max(0, c - w + 1)
        full = max(0, min(n, c + n - w + 1)) if w < c + n else 0      # tokens whose window is full
        pairs += full * w + (n - full) * c + (n - full) * (n - full + 1) // 2
    return keys, pairs


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] == "table":
        return {"bytes": 4 * case["n"] * case["R"], "flops": 20 * case["n"] * case["R"]}
    size = 4 if case.get("type") == "f32" else 2
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": 2 * size * n + 4 * case["T"] * (1 + min(case["R"], 8192 * case["R"] // case["T"])),
                "flops": 3 * case["T"] * case["H"] * case["R"]}
    if case["op"] == "qk":
        T, H, Hkv, D = (case[k] for k in ("T", "H", "Hkv", "D"))
        return {"bytes": T * (size * (H + 2 * Hkv) * D + size * H * D + 2 * 2 * Hkv * D + 12 + 4 * min(case["R"], 8192 * case["R"] // T)),
                "flops": T * (H + Hkv) * (4 * D + 3 * case["R"])}
    H, Hkv, D = (case[k] for k in ("H", "Hkv", "D"))
    keys, pairs = _visible(case)
    return {"bytes": 4 * keys * Hkv * D + case["tokens"] * H * (4 * D + 4), "flops": 4 * pairs * H * D}


def exact(case, seed):
    """The call's results in 64 bits from the definition."""
    s = prepare(case, seed)
    if case["op"] == "table":
        R, out = case["R"], torch.empty(case["n"], case["R"], device="cuda", dtype=torch.float64)
        pos = torch.arange(case["n"], device="cuda", dtype=torch.float64) + case["pos0"]
        # YaRN: pairs that turn over 32 times within the trained context keep their frequency, those that turn less than
        # once are slowed by the factor, between them it is blended pair by pair
        edge = [R / 2 * math.log(s["orig"] / (2 * math.pi * t), s["base"]) for t in (32.0, 1.0)]
        lo, hi = max(0, math.floor(edge[0])), min(R - 1, math.ceil(edge[1]))
        for i in range(R // 2):
            f = s["base"] ** (-i / (R / 2))
            if case["scaling"] == "linear":
                f /= case["factor"]
            elif case["scaling"] == "yarn":
                slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
                f *= 1.0 - slow + slow / case["factor"]
            out[:, i], out[:, R // 2 + i] = torch.cos(pos * f), torch.sin(pos * f)
        return out
    if case["op"] in ("rope", "qk"):
        R, off, D, H = case["R"], case["off"], case["D"], case["H"]
        pairs = [(2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + R // 2) for i in range(R // 2)]
        first = torch.tensor([off + a for a, _ in pairs], device="cuda")
        second = torch.tensor([off + b for _, b in pairs], device="cuda")
        c, sn = s["cs"][s["pos"].long()].double()[:, None, :].split(R // 2, -1)

        def turned(x, sign):
            y = x.clone()
            y[..., first] = x[..., first] * c - x[..., second] * (sign * sn)
            y[..., second] = x[..., second] * c + x[..., first] * (sign * sn)
            return y

        if case["op"] == "rope":
            return turned(s["x"].double().view(case["T"], H, D), -1.0 if case["inverse"] else 1.0)
        Hkv = case["Hkv"]
        q, k, v = s["qkv"].double().view(case["T"], -1, D).split([H, Hkv, Hkv], 1)
        if case["norm"]:
            q = q / (q.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["gq"].double()
            k = k / (k.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["gk"].double()
        kc, vc = s["kc"].double(), s["vc"].double()
        kc.view(-1, Hkv, D)[s["slot"]] = turned(k, 1.0)
        vc.view(-1, Hkv, D)[s["slot"]] = v
        return {"q": turned(q, 1.0), "k_cache": kc, "v_cache": vc}
    H, Hkv, D, bs = (case[k] for k in ("H", "Hkv", "D", "bs"))
    out = torch.empty(s["T"], H, D, device="cuda", dtype=torch.float64)
    lse = torch.empty(s["T"], H, device="cuda", dtype=torch.float64)
    start, length = s["start"].tolist(), s["ctx_len"].tolist()
    for b in range(case["B"]):
        n, L = start[b + 1] - start[b], length[b]
        if n == 0:
            continue
        at = torch.arange(L, device="cuda")
        rows = s["table"][b].long()[at // bs] * bs + at % bs
        p = L - n + torch.arange(n, device="cuda")
        sees = at[None, :] <= p[:, None]
        if case["window"]:
            sees &= at[None, :] > p[:, None] - case["window"]
        for h in range(H):
            k = s["kc"].view(-1, Hkv, D)[rows, h * Hkv // H].double()
            v = s["vc"].view(-1, Hkv, D)[rows, h * Hkv // H].double()
            x = (s["q"][start[b]:start[b + 1], h].double() @ k.t()) * s["scale"]
            x = torch.where(sees, x, torch.full_like(x, -math.inf))
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"][h].double().expand(n, 1)], 1)
            lse[start[b]:start[b + 1], h] = torch.logsumexp(x, 1)
            out[start[b]:start[b + 1], h] = torch.softmax(x, 1)[:, :L] @ v
    return {"out": out, "lse": lse}
