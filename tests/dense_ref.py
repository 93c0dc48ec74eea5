"""Plain 64-bit references of the dense-attention calls (rotary table, rotation, per-head norm + rotation + cache write,
attention over a paged cache) and the error bounds their tests use.  Torch in float64, on whatever device the inputs are.

Bounds.  A rounding to fp32 is off by at most 2^-24 of the value, to bf16 by 2^-8.
 rotation   x0 c - x1 s: two products and a sum, at most three fp32 roundings of parts no larger than |x0 c| + |x1 s|.
 norm       the D <= 256 squares are summed in at most 8 steps in a lane and 5 across lanes (14 roundings with the mean,
            16 with eps), halved by the root; the hardware's root is off by 2 ulps, 2^-22; with the three products behind
            it the factor is off by less than 8 + 4 + 3 = 15 of 2^-24, under 2^-20.
"""
import math
from decimal import Decimal, getcontext

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def pairs(R, half):
    return [(i, i + R // 2) if half else (2 * i, 2 * i + 1) for i in range(R // 2)]


def table(params, R, positions):
    """cos / sin rows of the given positions, from 60-digit decimals: [len(positions), R] float64."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    base, scaling, factor, orig, fast, slow, amplitude = params
    edge = lambda turns: R * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    if scaling == 2:
        lo, hi = max(math.floor(edge(fast)), 0), min(math.ceil(edge(slow)), R - 1)
    out = torch.empty(len(positions), R, dtype=torch.float64)
    for i in range(R // 2):
        f = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(R)).exp()
        if scaling == 1:
            f /= Decimal(factor)
        if scaling == 2:
            w = min(max(Decimal(i - lo) / max(Decimal(hi - lo), Decimal("0.001")), Decimal(0)), Decimal(1))
            f = f * (1 - w) + f / Decimal(factor) * w
        for r, p in enumerate(positions):
            turn = Decimal(int(p)) * f / two_pi
            a = float((turn - turn.to_integral_value()) * two_pi)
            out[r, i], out[r, R // 2 + i] = amplitude * math.cos(a), amplitude * math.sin(a)
    return out


def rotate(x, cs, R, off, half, inverse=False):
    """(rotated x, size of the parts each element is summed from); x [T, H, D] float64, cs [T, R]."""
    y, part = x.clone(), x.abs()
    if R:
        a = torch.tensor([off + p for p, _ in pairs(R, half)], device=x.device)
        b = torch.tensor([off + p for _, p in pairs(R, half)], device=x.device)
        c, s = cs.double()[:, None, :R // 2], cs.double()[:, None, R // 2:]
        s = -s if inverse else s
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        size = x[..., a].abs() * c.abs() + x[..., b].abs() * s.abs()
        part[..., a] = size
        part[..., b] = x[..., a].abs() * s.abs() + x[..., b].abs() * c.abs()
    return y, part


def norm(x, gamma, eps):
    x = x.double()
    return x if gamma is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()


def close(got, want, part, dtype, rel):
    """got (of dtype) within its own rounding and `rel` of the parts of want; equal where nothing is computed."""
    tol = HALF[dtype] * (want.abs() + rel * part) + rel * part
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())


def attention(q, k_rows, v_rows, new, lens, scale, causal, window, sink):
    """out [T, H, D], lse [T, H] and their bounds, from the definition, sequence by sequence.  q [T, H, D] holds the
    sequences' rows one after the other; k_rows[b], v_rows[b] [L, Hkv, D] the keys of sequence b (None: a masked key in
    its place is a row of NaN in `k_rows`, see `dead`).

    Bounds.  Score j is a sum of D products in fp32 by the tensor core: off by at most D 2^-23 of the sum of their
    magnitudes, and by 2^-22 of its size through the factor and the subtraction of the maximum: ds_j.  A weight
    e^(s_j - m) is off by ds_j + 2^-21 (the hardware's 2^x), its bf16 form by another 2^-8.  The denominator sums at most
    64 weights in a chain, then a tile at a time: 2^-24 for each step.  out is rounded once to bf16, 2^-8 of its value."""
    T, H, D = q.shape
    dev = q.device
    out, lse = torch.zeros(T, H, D, dtype=torch.float64, device=dev), torch.empty(T, H, dtype=torch.float64, device=dev)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for b, n in enumerate(new):
        n, L = int(n), int(lens[b])
        if n == 0:
            continue
        k, v, live = k_rows[b].double(), v_rows[b].double(), ~k_rows[b].isnan().all(-1).all(-1)
        k, v = torch.where(live[:, None, None], k, 0.0), torch.where(live[:, None, None], v, 0.0)
        Hkv = k.shape[1]
        qs = q[at:at + n].double().view(n, Hkv, H // Hkv, D)
        s = torch.einsum("nkgd,lkd->nkgl", qs, k) * scale
        size = torch.einsum("nkgd,lkd->nkgl", qs.abs(), k.abs()) * scale
        p = L - n + torch.arange(n, device=dev)
        j = torch.arange(L, device=dev)
        see = live[None, :].expand(n, L)
        if causal:
            see = see & (j[None, :] <= p[:, None])
        if window:
            see = see & (j[None, :] > p[:, None] - window)
        see = see[:, None, None, :]
        s = s.masked_fill(~see, -math.inf)
        sk = torch.full((H,), -math.inf, device=dev, dtype=torch.float64) if sink is None else sink.double()
        sk = sk.view(1, Hkv, H // Hkv, 1)
        m = torch.maximum(s.amax(-1, keepdim=True) if L else sk, sk).clamp(min=-1e300)
        w = (s - m).exp()
        den = w.sum(-1, keepdim=True) + (sk - m).exp()
        pr = torch.where(den > 0, w / den, 0.0)
        ds = ((D * 2.0 ** -23 + 2.0 ** -22) * size).masked_fill(~see, 0.0).amax(-1, keepdim=True) if L else 0 * den
        steps = (2 * 64 + L // 128 + 8) * 2.0 ** -24
        o = torch.einsum("nkgl,lkd->nkgd", pr, v)
        mean = torch.einsum("nkgl,lkd->nkgd", pr, v.abs())
        out[at:at + n] = o.reshape(n, H, D)
        out_tol[at:at + n] = ((2.0 ** -8 + 2 * ds + 2.0 ** -20 + steps) * 1.01 * mean + 2.0 ** -8 * o.abs()).reshape(n, H, D)
        le = torch.where(den > 0, m + den.log(), -math.inf)
        lse[at:at + n] = le.reshape(n, H)
        lse_tol[at:at + n] = (ds + steps + 2.0 ** -20 + 2.0 ** -22 * torch.where(den > 0, le.abs() + m.abs(), 0.0)).reshape(n, H)
        at += n
    return out, lse, out_tol, lse_tol
