"""Cases of the three calls that prepare the indexer's inputs, in a plain torch form and as calls of this library.

    norm   residual addition + RMS norm + E4M3 codes with one fp32 scale per 128 elements (dsa_add_rmsnorm_e4m3)
    gemm   projection of such codes by E4M3 weights with one scale per 128 x 128 block     (dsa_gemm_e4m3)
    slots  block tables, slot mapping and positions of a step from request lengths        (dsa_assign_slots)

A step of the sparse-attention layer runs them in this order of use: the request lengths give every new token its
cache slot and position; the hidden state is added to the residual stream, normalised and quantised; the projections
give the indexer's query rows (64 heads x 128), its shared key (128) and its head weights (64).

`own` chooses between the plain form (False) and the library's calls (True).
"""
import math

import torch

own = False

GROUP = 128          # elements per activation scale, and rows / columns per weight scale
FP8_MAX = 448.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


_calls = None


def _lib():
    global _calls
    if _calls is None:
        from deepseek_v4_sparse_dsa_gb300 import dsa
        _calls = dsa
    return _calls


def _groups(n):
    return -(-n // GROUP)


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one sequence: nothing but latency
        {"name": "norm 1x4096", "op": "norm", "T": 1, "D": 4096, "pad": 0, "type": "bf16", "residual": True, "y": False, "pow2": False},
        # the decode batch of 64 sequences, with power-of-two scales and the normalised row kept in bf16 too
        {"name": "norm 64x2048 pow2", "op": "norm", "T": 64, "D": 2048, "pad": 0, "type": "bf16", "residual": True, "y": True, "pow2": True},
        # an odd batch of a width that fills neither its last group nor whole 16-byte pieces, cut out of a wider tensor
        {"name": "norm 517x4999 f32", "op": "norm", "T": 517, "D": 4999, "pad": 3, "type": "f32", "residual": False, "y": True, "pow2": False},
        # the 16K prefill
        {"name": "norm 16384x4096", "op": "norm", "T": 16384, "D": 4096, "pad": 0, "type": "bf16", "residual": True, "y": False, "pow2": False},
        # the indexer's query projection (64 heads x 128) for one token: the weights are read once
        {"name": "gemm 1x8192x2048", "op": "gemm", "M": 1, "N": 8192, "K": 2048, "out": "bf16"},
        # the same projection for a decode batch of 64 sequences
        {"name": "gemm 64x8192x4096", "op": "gemm", "M": 64, "N": 8192, "K": 4096, "out": "bf16"},
        # a ragged batch: no size is a whole number of tiles or blocks
        {"name": "gemm 333x1000x1808", "op": "gemm", "M": 333, "N": 1000, "K": 1808, "out": "f32"},
        # the head weights (64 of them, fp32) of a chunk of 8192 query tokens
        {"name": "gemm 8192x64x4096", "op": "gemm", "M": 8192, "N": 64, "K": 4096, "out": "f32"},
        # the query projection of a chunk of 8192 query tokens: bound by the tensor cores
        {"name": "gemm 8192x8192x4096", "op": "gemm", "M": 8192, "N": 8192, "K": 4096, "out": "bf16"},
        # a decode step: 64 sequences, one new token each, contexts up to 64K
        {"name": "slots 64x1", "op": "slots", "B": 64, "bs": 64, "ctx": 65536, "tokens": 64, "each": 1},
        # a mixed step: 1000 requests share 8192 new tokens unevenly, some have none
        {"name": "slots 1000 mixed", "op": "slots", "B": 1000, "bs": 16, "ctx": 5000, "tokens": 8192, "each": 0},
        # long prompts: 32 requests bring 256K tokens
        {"name": "slots 32 prompts", "op": "slots", "B": 32, "bs": 64, "ctx": 1000, "tokens": 262144, "each": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "slots"])
    if op == "norm":
        D = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            D = max(8, D // 8 * 8)
        T = _log(rng, 1, max(1, min(16384, 16384 * 4096 // D)))
        typ = rng.choice(["bf16", "bf16", "f32"])
        if typ == "f32":
            T = max(1, T // 4)
        return {"op": op, "T": T, "D": D, "pad": rng.choice([0, 0, 1, 8, 24]), "type": typ, "residual": rng.random() < 0.6,
                "y": rng.random() < 0.4, "pow2": T * _groups(D) <= 2048 and rng.random() < 0.5}
    if op == "gemm":
        K = 16 * _log(rng, 4, 512)
        N = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            N = max(64, N // 64 * 64)
        M = _log(rng, 1, max(1, min(16384, 8192 * 8192 * 4096 // (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "f32"])}
    B = _log(rng, 1, 4096)
    bs = rng.choice([8, 16, 20, 32, 64, 64, 128, 256])
    ctx = _log(rng, 16, max(16, min(131072, 4000000 * bs // B)))
    if rng.random() < 0.5:
        each = rng.choice([1, 1, 2, 3, 4])
        return {"op": op, "B": B, "bs": bs, "ctx": ctx, "tokens": B * each + rng.choice([0, 0, 5]), "each": each}
    return {"op": op, "B": B, "bs": bs, "ctx": ctx, "tokens": _log(rng, B, max(B, min(262144, 4000000 * bs // B))), "each": 0}


# ------------------------------------------------------------------------------------------------ inputs

def _quantise(x):
    """E4M3 codes of x [..., 128] and the scale amax / 448 of each group."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    return (x / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), scale.squeeze(-1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        T, D, typ = case["T"], case["D"], TYPES[case["type"]]
        ld = D + case["pad"]
        # a few channels of a hidden state are far larger than the rest
        chan = 1.0 + 20.0 * (torch.rand(D, generator=g, device=dev) < 0.01)
        # rows of a wider tensor, `ld` elements apart
        s["x"] = torch.zeros(T, ld, device=dev, dtype=typ)[:, :D]
        s["x"].copy_((randn(T, D) * chan).to(typ))
        s["res"] = None
        if case["residual"]:
            s["res"] = (randn(T, D) * chan * 3.0).to(typ)
            s["res_out"] = torch.empty(T, D, device=dev, dtype=typ)
        s["gamma"] = 1.0 + 0.1 * randn(D)
        s["y"] = torch.empty(T, D, device=dev, dtype=typ) if case["y"] else None
        s["codes"] = torch.empty(T, D, device=dev, dtype=torch.float8_e4m3fn)
        s["scale"] = torch.empty(T, _groups(D), device=dev)
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        gk, gn = _groups(K), _groups(N)
        a = torch.zeros(M, gk * GROUP, device=dev)
        a[:, :K] = randn(M, K)
        a, s["a_scale"] = _quantise(a.view(M, gk, GROUP))
        s["a"] = a.view(M, gk * GROUP)[:, :K].contiguous()
        w = torch.zeros(gn * GROUP, gk * GROUP, device=dev)
        w[:N, :K] = randn(N, K) * 0.02
        w = w.view(gn, GROUP, gk, GROUP).transpose(1, 2).reshape(gn, gk, GROUP * GROUP)
        w, s["w_scale"] = _quantise(w)
        s["w"] = w.view(gn, gk, GROUP, GROUP).transpose(1, 2).reshape(gn * GROUP, gk * GROUP)[:N, :K].contiguous()
        s["out_buf"] = torch.empty(M, N, device=dev, dtype=TYPES[case["out"]])
    else:
        B, bs, ctx, tokens, each = (case[k] for k in ("B", "bs", "ctx", "tokens", "each"))
        s["cached"] = torch.randint(0, ctx, (B,), generator=g, device=dev, dtype=torch.int32)
        if each:
            s["new"] = torch.full((B,), each, device=dev, dtype=torch.int32)
            longest = each
        else:
            # uneven shares of the step's tokens, a fifth of the requests without any
            share = torch.rand(B, generator=g, device=dev, dtype=torch.float64) ** 4
            share *= torch.rand(B, generator=g, device=dev) < 0.8
            s["new"] = (share / share.sum().clamp(min=1e-9) * tokens).floor().to(torch.int32)
            longest = tokens
        stride = -(-(ctx + longest) // bs)
        n_free = tokens // bs + B + 1
        held = B * -(-ctx // bs)
        pool = torch.randperm(held + n_free, generator=g, device=dev, dtype=torch.int32)
        table = torch.full((B, stride), -1, device=dev, dtype=torch.int32)
        table[:, : -(-ctx // bs)] = pool[:held].view(B, -1)
        cols = torch.arange(stride, device=dev)
        table.masked_fill_(cols[None, :] >= ((s["cached"] + bs - 1) // bs)[:, None], -1)
        s.update(table=table, free=pool[held:].clone(), num_blocks=held + n_free,
                 context=torch.empty(B, device=dev, dtype=torch.int32),
                 start=torch.empty(B + 1, device=dev, dtype=torch.int32),
                 slot=torch.empty(tokens, device=dev, dtype=torch.int64),
                 pos=torch.empty(tokens, device=dev, dtype=torch.int32),
                 used=torch.empty(1, device=dev, dtype=torch.int32))
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return {"norm": _norm, "gemm": _gemm, "slots": _slots}[s["op"]](s)


def _norm(s):
    T, D = s["T"], s["D"]
    if own:
        dsa = _lib()
        typ = dsa.DSA_REAL_F32 if s["type"] == "f32" else dsa.DSA_REAL_BF16
        dsa.dsa_add_rmsnorm_e4m3(s["x"], s["x"].stride(0), s["res"], D, s["gamma"], EPS, T, D, typ, s.get("res_out"),
                                 s["y"], s["codes"], D, s["scale"], s["pow2"])
        return {"residual": s.get("res_out"), "y": s["y"], "codes": s["codes"], "scale": s["scale"]}
    r = s["x"]
    if s["res"] is not None:
        r = (r.float() + s["res"].float()).to(r.dtype)
    v = r.float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["gamma"]
    n = _groups(D)
    z = torch.nn.functional.pad(y, (0, n * GROUP - D)).view(T, n, GROUP)
    amax = z.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    if s["pow2"]:
        m, e = torch.frexp(scale)      # scale = m 2^e, 1/2 <= m < 1: the next power of two at or above it
        scale = torch.ldexp(torch.ones_like(scale), torch.where(m == 0.5, e - 1, e))
    codes = (z / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return {"residual": r if s["res"] is not None else None, "y": y.to(s["x"].dtype) if s["y"] is not None else None,
            "codes": codes.view(T, n * GROUP)[:, :D], "scale": scale}


def _gemm(s):
    M, N, K = s["M"], s["N"], s["K"]
    if own:
        dsa = _lib()
        typ = dsa.DSA_REAL_F32 if s["out"] == "f32" else dsa.DSA_REAL_BF16
        dsa.dsa_gemm_e4m3(s["a"], K, s["a_scale"], s["w"], K, s["w_scale"], M, N, K, s["out_buf"], N, typ)
        return s["out_buf"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(GROUP, 1)[:, :K]
    w = s["w"].float() * s["w_scale"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    return (a @ w.t()).to(TYPES[s["out"]])


def _slots(s):
    B, bs, tokens = s["B"], s["bs"], s["tokens"]
    if own:
        dsa = _lib()
        dsa.dsa_assign_slots(s["cached"], s["new"], B, bs, s["free"], s["free"].shape[0], s["num_blocks"], s["table"],
                             s["table"].shape[1], tokens, s["context"], s["start"], s["slot"], s["pos"], s["used"])
        return {"table": s["table"], "context": s["context"], "start": s["start"], "slot": s["slot"], "pos": s["pos"],
                "used": s["used"]}
    cached, new, free, table = s["cached"], s["new"], s["free"], s["table"]
    context = cached + new
    ends = torch.cumsum(new, 0, dtype=torch.int32)
    start = torch.nn.functional.pad(ends, (1, 0))
    have = (cached + (bs - 1)) // bs                        # pages held before the step, and pages it adds
    need = (context + (bs - 1)) // bs - have
    total = torch.cumsum(need, 0, dtype=torch.int32)
    first = total - need                                     # the request's first entry of the free list
    col = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    table.copy_(torch.where(fresh, free[(first[:, None] + col).clamp(0, free.shape[0] - 1)], table))
    t = torch.arange(tokens, device=table.device, dtype=torch.int32)
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    live = t < ends[-1]
    pos = torch.where(live, cached[b] + t - start[b], 0)
    slot = torch.where(live, table[b, pos // bs].long() * bs + pos % bs, -1)
    return {"table": table, "context": context, "start": start, "slot": slot, "pos": pos, "used": total[-1:]}


# ------------------------------------------------------------------------------------------------ floor and exact values

def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        size = 4 if case["type"] == "f32" else 2
        words = 1 + (2 if case["residual"] else 0) + (1 if case["y"] else 0)
        return {"bytes": T * D * (size * words + 1) + 4 * T * _groups(D) + 4 * D, "flops": 8 * T * D}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": M * K + N * K + 4 * _groups(K) * (M + _groups(N)) + size * M * N, "flops": 2 * M * N * K}
    B, tokens = case["B"], case["tokens"]
    pages = tokens // case["bs"] + (B if case["each"] else 0) / case["bs"]
    # lengths in, lengths and starts out; slot and position of each token; a free-list entry read and a table entry
    # written per new page, and the last page of each request read
    return {"bytes": 16 * B + 12 * tokens + 8 * pages + 4 * min(B, tokens), "flops": 8 * tokens}


def exact(case, seed):
    """The call's results in 64 bits from the definition; None for the whole numbers of `slots`."""
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    if case["op"] == "gemm":
        K = case["K"]
        out = torch.zeros(case["M"], case["N"], device=s["a"].device, dtype=torch.float64)
        col = torch.arange(case["N"], device=out.device) // GROUP
        for k0 in range(0, K, GROUP):                     # sum over the blocks of K of (codes . codes) x both scales
            part = s["a"][:, k0:k0 + GROUP].double() @ s["w"][:, k0:k0 + GROUP].double().t()
            out += part * s["a_scale"][:, k0 // GROUP, None].double() * s["w_scale"][col, k0 // GROUP].double()[None, :]
        return out
    T, D = case["T"], case["D"]
    if T * D > 1 << 26:
        return None
    r = s["x"].double()
    if s["res"] is not None:
        r = (r + s["res"].double()).to(s["x"].dtype).double()      # the residual stream is held in its own type
    y = r / (r.square().sum(-1, keepdim=True) / D + EPS).sqrt() * s["gamma"].double()
    scale = torch.ones(T, _groups(D), device=y.device, dtype=torch.float64)
    codes = torch.empty_like(y)
    for j in range(_groups(D)):
        part = y[:, j * GROUP:(j + 1) * GROUP]
        amax = part.abs().amax(-1)
        live = amax > 0
        scale[live, j] = amax[live] / FP8_MAX
        if case["pow2"]:
            scale[:, j] = torch.exp2(torch.ceil(torch.log2(scale[:, j])))
        q = (part / scale[:, j:j + 1]).abs()
        # E4M3: three mantissa bits, exponents down to 2^-6, ties to the even code
        step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
        codes[:, j * GROUP:(j + 1) * GROUP] = torch.sign(part) * (torch.round(q / step) * step).clamp(max=FP8_MAX)
    return {"residual": r if s["res"] is not None else None, "y": y if s["y"] is not None else None,
            "codes": codes, "scale": scale}
