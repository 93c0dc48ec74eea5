"""Plain 64-bit references of the calls that prepare a step's inputs (numpy, loops where the
definition is a loop), and the error bounds their tests use."""
import numpy as np

E4M3_VALUES = None


def e4m3_values():
    """The 256 E4M3 codes' values (NaN for 0x7F, 0xFF)."""
    global E4M3_VALUES
    if E4M3_VALUES is None:
        v = np.empty(256)
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            v[c] = (-1.0 if c & 128 else 1.0) * (np.nan if e == 15 and m == 7 else x)
        E4M3_VALUES = v
    return E4M3_VALUES


def bf16_round(x):
    """float64 -> nearest-even bf16 value (as float64), by way of fp32 bits."""
    f = np.asarray(x, np.float64)
    m, e = np.frexp(f)                                   # f = m 2^e, 1/2 <= |m| < 1: 8 significant bits
    e = np.maximum(e, -125)
    return np.where(np.isfinite(f), np.rint(np.ldexp(f, 8 - e)) * np.ldexp(1.0, e - 8), f)


def assign_slots(cached, new, bs, free, num_blocks, table, max_tokens):
    """(table, context, start, slots, positions, used) by the definition, one token at a time.  Valid inputs."""
    table = table.copy()
    B = len(cached)
    context = cached + new
    start = np.zeros(B + 1, np.int64)
    slots = np.full(max_tokens, -1, np.int64)
    pos = np.zeros(max_tokens, np.int64)
    used = t = 0
    for b in range(B):
        have, want = -(-int(cached[b]) // bs), -(-int(context[b]) // bs)
        for page in range(have, want):
            table[b, page] = free[used]
            used += 1
        for p in range(int(cached[b]), int(context[b])):
            blk = int(table[b, p // bs])
            assert 0 <= blk < num_blocks
            slots[t], pos[t] = blk * bs + p % bs, p
            t += 1
        start[b + 1] = t
    return table, context, start, slots, pos, used


def add_rmsnorm(x, res, gamma, eps, bf16):
    """(r, y) in float64: r rounded once to the input's type, y unrounded."""
    r = np.asarray(x, np.float64)
    if res is not None:
        s = r + np.asarray(res, np.float64)
        r = bf16_round(s) if bf16 else s.astype(np.float32).astype(np.float64)
    return r, r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


# Relative error of y before its rounding: each thread sums up to 32 squares, a warp 5 levels and up to
# 32 warps' sums are added: at most 69 roundings of 2^-24, halved by the root; the mean, eps, root and the
# two products add 5 more.  40 * 2^-24 covers it; 2^-18 = 64 * 2^-24 is used.
Y_REL = 2.0 ** -18


def check_quantised(y, codes, scale, pow2):
    """codes, scale [.., groups] against y (float64) by the definition, allowing y's fp32 error."""
    T, D = y.shape
    G = -(-D // 128)
    vals = e4m3_values()[codes]
    assert scale.shape == (T, G) and np.isfinite(vals).all()
    for g in range(G):
        part, q = y[:, g * 128:(g + 1) * 128], vals[:, g * 128:(g + 1) * 128]
        s = scale[:, g].astype(np.float64)
        want = np.abs(part).max(-1) / 448.0
        zero = want == 0
        assert (s[zero] == 1.0).all() and (q[zero] == 0).all()
        want = np.maximum(want, 2.0 ** -126)[~zero]
        s1 = s[~zero]
        if pow2:
            assert (np.frexp(s1)[0] == 0.5).all()
            assert (s1 >= want * (1 - 2 * Y_REL)).all() and (s1 < 2 * want * (1 + 2 * Y_REL)).all()
        else:
            assert (np.abs(s1 - want) <= 2 * Y_REL * want).all()
        ratio = np.abs(part[~zero] / s1[:, None])
        # half a step: 2^-4 relative for normal codes, 2^-10 below 2^-6
        tol = np.maximum(ratio * 2.0 ** -4, 2.0 ** -10) + 2 * Y_REL * ratio
        assert (np.abs(q[~zero] - part[~zero] / s1[:, None]) <= tol).all()


def gemm(a, a_scale, w, w_scale):
    """(out, bound): the block-scaled product of codes in float64, and how far fp32 may leave it.

    The bound: a block's 128 products are exact in fp32 and summed with at most 127 roundings, taken as
    2^-23 each (truncation counted); its two scales' product, the multiplication and the sums over the
    blocks and up to 8 parts round at 2^-24 each, relative to the sum of the terms' magnitudes."""
    vals = e4m3_values()
    A, W = vals[a], vals[w]
    M, K = A.shape
    N = W.shape[0]
    G = -(-K // 128)
    out, mag = np.zeros((M, N)), np.zeros((M, N))
    for kb in range(G):
        k = slice(kb * 128, min(K, kb * 128 + 128))
        s = a_scale[:, kb].astype(np.float64)[:, None] * np.repeat(w_scale[:, kb].astype(np.float64), 128)[None, :N]
        out += (A[:, k] @ W[:, k].T) * s
        mag += (np.abs(A[:, k]) @ np.abs(W[:, k]).T) * np.abs(s)
    return out, mag * (127 * 2.0 ** -23 + (G + 8 + 2) * 2.0 ** -24)
