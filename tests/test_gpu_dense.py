"""The dense-attention calls on the GPU against plain 64-bit references (dense_ref.py, where the bounds are derived)."""
import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from deepseek_v4_sparse_dsa_gb300 import dsa  # noqa: E402

BF16, F32 = dsa.DSA_REAL_BF16, dsa.DSA_REAL_F32
TYPE = {torch.bfloat16: BF16, torch.float32: F32}
INTER, HALF = dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cos_sin(n, R, seed=0, shift=0):
    """Any table will do for the rotation: random angles; `shift` elements off a 16-byte boundary."""
    a = torch.rand(n, R // 2, device="cuda", generator=gen(seed)) * 6.28
    t = torch.empty(n * R + shift, device="cuda")[shift:].view(n, R)
    return t.copy_(torch.cat([a.cos(), a.sin()], 1))


# ------------------------------------------------------------------ table
@pytest.mark.parametrize("R", [2, 6, 64, 128, 250, 256])
@pytest.mark.parametrize("params", [(10000.0, 0, 1.0, 4096.0, 32.0, 1.0, 1.0), (500000.0, 1, 8.0, 4096.0, 32.0, 1.0, 1.0),
                                    (10000.0, 2, 40.0, 4096.0, 32.0, 1.0, 1.2689), (1.5, 2, 16.0, 100.0, 4.0, 4.0, 0.5)])
def test_table(R, params):
    # 0.7: near a quarter turn; 2^31 - 1 is the last position there is
    for pos0, n in [(0, 1), (0, 37), (4090, 9), ((1 << 20) - 3, 5), ((1 << 31) - 3, 3)]:
        out = torch.full((n + 1, R), -7.0, device="cuda")
        dsa.dsa_rope_table(dsa.make_rope_params(*params), R, pos0, n, out)
        want = ref.table(params, R, range(pos0, pos0 + n))
        assert bool((out[n] == -7.0).all())
        assert float((out[:n].cpu().double() - want).abs().max()) <= 2.0 ** -22 * params[-1]
    assert dsa.dsa_device_error() == 0


def test_table_many_rows():
    # more rows than one pass of the grid: the phase is carried from row to row
    n, R = 300001, 14
    out = torch.empty(n, R, device="cuda")
    dsa.dsa_rope_table(dsa.make_rope_params(), R, 12345, n, out)
    at = [0, 1, 7, 40000, 123456, 299999, 300000]
    want = ref.table((10000.0, 0, 1.0, 4096.0, 32.0, 1.0, 1.0), R, [12345 + r for r in at])
    assert float((out[at].cpu().double() - want).abs().max()) <= 2.0 ** -22
    near = out.double()
    assert bool(((near[:, :R // 2] ** 2 + near[:, R // 2:] ** 2 - 1).abs() <= 2.0 ** -21).all())


def test_table_feeds_the_indexer_query():
    # the same layout as dsa_indexer_q_rope_quant reads: its codes times its scales are the rotated query
    T, H, R = 9, 64, 64
    cs = torch.empty(4096, R, device="cuda")
    dsa.dsa_rope_table(dsa.make_rope_params(scaling=dsa.DSA_ROPE_YARN, factor=4.0, original_max_pos=1024.0), R, 0, 4096, cs)
    q = torch.randn(T, H, 128, device="cuda", generator=gen(1)).bfloat16()
    pos = torch.randint(0, 4096, (T,), device="cuda", generator=gen(2), dtype=torch.int32)
    codes = torch.empty(T, H, 128, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.empty(T, H, device="cuda")
    dsa.dsa_indexer_q_rope_quant(q, pos, cs, 4096, R, T, H, 128, codes, scale)
    y = torch.empty_like(q, dtype=torch.float32)
    dsa.dsa_rope(q.float(), H * 128, 128, pos, cs, 4096, R, 0, INTER, False, T, H, 128, F32, y, H * 128, 128)
    # half an E4M3 step: 2^-4 of the value, or of the smallest normal 2^-6
    tol = (y.abs() * 2.0 ** -4).clamp(min=2.0 ** -10 * float(scale.max())) * (1 + 2.0 ** -20)
    assert bool(((codes.float() * scale[..., None] - y).abs() <= tol).all())
    assert dsa.dsa_device_error() == 0


# ------------------------------------------------------------------ rotation
SHAPES = [  # T, H, D, R, off
    (1, 1, 2, 2, 0), (3, 2, 8, 8, 0), (5, 3, 64, 64, 0), (70, 64, 128, 64, 64), (33, 5, 128, 128, 0), (9, 4, 128, 64, 32),
    (7, 3, 96, 32, 20), (4, 2, 192, 64, 128), (6, 2, 256, 256, 0), (2, 1, 256, 8, 4), (11, 3, 80, 40, 40), (5, 2, 128, 4, 0),
    (8, 3, 7, 4, 1), (3, 5, 129, 100, 17), (2, 2, 255, 254, 1), (700, 9, 40, 16, 8),
]


def rope_case(T, H, D, R, off, dtype, layout, inverse, pad=0, hpad=0, shift=0, seed=0):
    ldx, hx = H * (D + hpad) + pad, D + hpad
    x0 = torch.randn(T * ldx + shift, device="cuda", generator=gen(seed)).to(dtype)
    x = torch.as_strided(x0, (T, H, D), (ldx, hx, 1), shift)
    cs = cos_sin(50, R, seed + 1)
    pos = torch.randint(0, 50, (T,), device="cuda", generator=gen(seed + 2), dtype=torch.int32)
    want, part = ref.rotate(x.double(), cs[pos.long()], R, off, layout == HALF, inverse)
    return x0, x, ldx, hx, cs, pos, want, part


@pytest.mark.parametrize("layout", [INTER, HALF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(shape, dtype, layout):
    T, H, D, R, off = shape
    for inverse, pad, hpad, shift in [(False, 0, 0, 0), (True, 8, 8, 0), (False, 4, 4, 4), (True, 5, 3, 1)]:
        x0, x, ldx, hx, cs, pos, want, part = rope_case(T, H, D, R, off, dtype, layout, inverse, pad, hpad, shift)
        y0 = torch.full((T * ldx + shift,), -7.0, device="cuda", dtype=dtype)
        y = torch.as_strided(y0, (T, H, D), (ldx, hx, 1), shift)
        dsa.dsa_rope(x, ldx, hx, pos, cs, 50, R, off, layout, inverse, T, H, D, TYPE[dtype], y, ldx, hx)
        ref.close(y, want, part, dtype, 3 * 2.0 ** -24)
        assert torch.equal(y[..., :off], x[..., :off]) and torch.equal(y[..., off + R:], x[..., off + R:])
        y.fill_(-7.0)
        assert bool((y0 == -7.0).all())                    # nothing between the heads is written
        keep = x0.clone()
        torch.as_strided(keep, (T, H, D), (ldx, hx, 1), shift).copy_(want)
        dsa.dsa_rope(x, ldx, hx, pos, cs, 50, R, off, layout, inverse, T, H, D, TYPE[dtype], x, ldx, hx)   # in place
        ref.close(x, want, part, dtype, 3 * 2.0 ** -24)
        x.copy_(torch.as_strided(keep, (T, H, D), (ldx, hx, 1), shift))
        assert torch.equal(x0, keep)
    assert dsa.dsa_device_error() == 0


def test_rope_head_major_and_unaligned_table():
    # [H, T, D]: heads far apart, tokens side by side; a table that starts 4 bytes off a 16-byte boundary
    T, H, D, R = 19, 6, 128, 64
    x = torch.randn(H, T, D, device="cuda", generator=gen(3))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    for shift in (0, 1):
        cs = cos_sin(T, R, 4, shift)
        y = torch.empty(T, H, D, device="cuda")
        dsa.dsa_rope(x, D, T * D, pos, cs, T, R, 32, HALF, False, T, H, D, F32, y, H * D, D)
        want, part = ref.rotate(x.transpose(0, 1).double(), cs, R, 32, True)
        ref.close(y, want, part, torch.float32, 3 * 2.0 ** -24)
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("off", [0, 3])
def test_rope_bad_positions(off):
    T, H, D, R = 5, 3, 24, 16
    x = torch.randn(T, H, D, device="cuda", generator=gen(5))
    cs = cos_sin(10, R)
    pos = torch.tensor([0, -1, 9, 10, 2147483647], device="cuda", dtype=torch.int32)
    y = torch.empty_like(x)
    dsa.dsa_rope(x, H * D, D, pos, cs, 10, R, off, HALF, False, T, H, D, F32, y, H * D, D)
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    want, part = ref.rotate(x.double(), cs[pos.clamp(0, 9).long()], R, off, True)
    for t in (1, 3, 4):
        want[t, :, off:off + R] = 0
        part[t, :, off:off + R] = 0
    ref.close(y, want, part, torch.float32, 3 * 2.0 ** -24)


def test_rope_inverse_is_the_gradient():
    # y = R x: the gradient of sum(g y) is R^T g, against the formula and against differences
    T, H, D, R = 4, 2, 16, 12
    x, g = (torch.randn(T, H, D, device="cuda", generator=gen(s)) for s in (6, 7))
    cs, pos = cos_sin(8, R), torch.tensor([0, 3, 7, 1], device="cuda", dtype=torch.int32)
    call = lambda v, inv: dsa.dsa_rope(v, H * D, D, pos, cs, 8, R, 2, INTER, inv, T, H, D, F32, out, H * D, D)  # noqa: E731
    out = torch.empty_like(x)
    call(g, True)
    grad = out.clone()
    leaf = x.double().requires_grad_(True)
    (ref.rotate(leaf, cs[pos.long()], R, 2, False)[0] * g.double()).sum().backward()
    _, part = ref.rotate(g.double(), cs[pos.long()], R, 2, False, True)
    ref.close(grad, leaf.grad, part, torch.float32, 3 * 2.0 ** -24)
    d = torch.randn(T, H, D, device="cuda", generator=gen(8))
    call(x + d, False)
    up = (out.double() * g.double()).sum()
    call(x - d, False)
    slope = (up - (out.double() * g.double()).sum()) / 2
    size = float((d.double().abs() + x.double().abs()).sum() * g.abs().max())
    assert abs(float(slope - (grad.double() * d.double()).sum())) <= 2.0 ** -21 * size


# ------------------------------------------------------------------ norm, rotation, cache
class QK:
    def __init__(self, T, H, Hkv, D, R, off, layout, dtype, bs=16, norm=True, fused=True, head_major=False, values=True,
                 seed=0, shift=0, slots=None):
        g = gen(seed)
        self.__dict__.update(T=T, H=H, Hkv=Hkv, D=D, R=R, off=off, layout=layout, dtype=dtype, bs=bs)
        width = (H + 2 * Hkv) * D
        self.ld = width + (0 if fused else 3)
        store = torch.randn(T * self.ld + shift, device="cuda", generator=g).mul_(3).to(dtype)
        x = torch.as_strided(store, (T, width), (self.ld, 1), shift)
        self.q, self.k, self.v = x[:, :H * D], x[:, H * D:(H + Hkv) * D], x[:, (H + Hkv) * D:]
        self.values = values
        self.gq = torch.randn(D, device="cuda", generator=g) if norm else None
        self.gk = torch.randn(D, device="cuda", generator=g) if norm else None
        self.cs = cos_sin(40, R, seed + 1) if R else None
        self.pos = torch.randint(0, 40, (T,), device="cuda", generator=g, dtype=torch.int32)
        self.blocks = -(-T // bs) + 1
        shape = (self.blocks, Hkv, bs, D) if head_major else (self.blocks, bs, Hkv, D)
        self.kc, self.vc = (torch.randn(shape, device="cuda", generator=g).bfloat16() for _ in range(2))
        if head_major:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.slot = torch.randperm(self.blocks * bs, device="cuda", generator=g)[:T].contiguous() if slots is None else slots
        self.kc0, self.vc0 = self.kc.clone(), self.vc.clone()

    def run(self, q_out=None, k_out=None, cache=True, stream=None):
        T, H, Hkv, D = self.T, self.H, self.Hkv, self.D
        self.qo = torch.empty(T, H * D, device="cuda", dtype=self.dtype) if q_out is None else q_out
        self.ko = k_out
        kv = dsa.make_kv_cache(self.kc, self.vc if self.values else None) if cache else dsa.make_kv_cache(None)
        dsa.dsa_qk_norm_rope(self.q, self.ld, H, self.k, self.ld, Hkv, self.v if self.values else None, self.ld, T, D,
                             TYPE[self.dtype], self.gq, self.gk, 1e-5, self.pos if self.R else None, self.cs,
                             40 if self.R else 0, self.R, self.off, self.layout, self.qo, self.qo.stride(0), k_out,
                             0 if k_out is None else k_out.stride(0), kv, self.slot if cache else None, stream)

    def want(self):
        T, D = self.T, self.D
        cs = self.cs[self.pos.long()] if self.R else None
        q = ref.norm(self.q.reshape(T, -1, D), self.gq, 1e-5) if self.H else self.q.reshape(T, 0, D).double()
        k = ref.norm(self.k.reshape(T, -1, D), self.gk, 1e-5)
        return [ref.rotate(a.double(), cs, self.R, self.off, self.layout == HALF) for a in (q, k)]

    def check(self, wanted, cache=True):
        T, D, Hkv = self.T, self.D, self.Hkv
        rel = 2.0 ** -20 + 3 * 2.0 ** -24 if self.gq is not None else 3 * 2.0 ** -24
        (q, qp), (k, kp) = wanted
        if self.H:
            ref.close(self.qo.reshape(T, -1, D), q, qp, self.dtype, rel)
        if self.ko is not None:
            ref.close(self.ko.reshape(T, -1, D), k, kp, self.dtype, rel)
        if cache:
            on = (self.slot >= 0) & (self.slot < self.blocks * self.bs)
            s = self.slot[on]
            b, r = s // self.bs, s % self.bs
            ref.close(self.kc[b, r], k[on], kp[on], torch.bfloat16, rel)
            if self.values:
                assert torch.equal(self.vc[b, r], self.v.reshape(T, -1, D)[on].bfloat16())
            # every other row of the cache stays as it was
            self.kc[b, r] = self.kc0[b, r]
            if self.values:
                self.vc[b, r] = self.vc0[b, r]
        assert torch.equal(self.kc, self.kc0) and torch.equal(self.vc, self.vc0)


QKS = [  # T, H, Hkv, D, R, off
    (1, 64, 8, 128, 128, 0), (65, 8, 2, 64, 64, 0), (33, 7, 1, 80, 40, 40), (130, 6, 3, 128, 64, 64), (5, 1, 1, 256, 128, 64),
    (3, 2, 2, 192, 64, 128), (9, 3, 1, 8, 8, 0), (17, 5, 5, 96, 24, 12), (4, 3, 3, 33, 10, 7), (2, 64, 64, 128, 32, 0),
    (6, 2, 1, 2, 2, 0), (8, 4, 2, 128, 0, 0), (700, 4, 1, 128, 64, 64), (12, 0, 4, 64, 32, 0), (12, 4, 1, 251, 250, 1),
]


@pytest.mark.parametrize("layout", [INTER, HALF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", QKS)
def test_qk_norm_rope(shape, dtype, layout):
    for i, kw in enumerate([dict(), dict(norm=False, bs=1), dict(fused=False, bs=20, shift=1), dict(head_major=True, bs=64)]):
        c = QK(*shape, layout, dtype, seed=10 * i, **kw)
        wanted = c.want()
        c.run(k_out=torch.empty(c.T, c.Hkv * c.D, device="cuda", dtype=dtype) if i % 2 else None)
        c.check(wanted)
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("D", [128, 67])
def test_qk_norm_rope_in_place_keys_only_and_no_cache(D):
    R = 64
    c = QK(21, 6, 2, D, R, 2, HALF, torch.bfloat16)
    wanted, v = c.want(), c.v.clone()
    c.run(q_out=c.q, k_out=c.k, cache=False)               # within the projection's own output
    c.check(wanted, cache=False)
    assert torch.equal(c.v, v)
    c = QK(21, 6, 2, D, R, 2, INTER, torch.bfloat16, values=False, seed=1)
    wanted = c.want()
    c.run()
    c.check(wanted)
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("D", [64, 30])
def test_qk_norm_rope_slots_that_are_none(D):
    bs = 4
    slots = torch.tensor([3, -1, 11, -5, 12, 2 ** 40, 0], device="cuda")     # the pool has 3 blocks of 4 rows
    c = QK(7, 2, 2, D, 16, 0, HALF, torch.float32, bs=bs, slots=slots)
    c.blocks = 3
    c.kc, c.vc = c.kc[:3].contiguous(), c.vc[:3].contiguous()
    c.kc0, c.vc0 = c.kc.clone(), c.vc.clone()
    wanted = c.want()
    c.run()
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    c.check(wanted)
    c.slot = torch.full((7,), -1, device="cuda")
    c.run()                                                # padding alone is no error
    assert dsa.dsa_device_error() == 0
    c.check(wanted)


@pytest.mark.parametrize("D", [128, 20])
def test_qk_norm_rope_bad_positions(D):
    c = QK(6, 3, 1, D, 16, 4, INTER, torch.float32)
    c.pos[1], c.pos[4] = -3, 40
    good = c.pos.clone()
    c.pos.clamp_(0, 39)
    wanted = c.want()
    for w, p in wanted:
        for a in (w, p):
            a[[1, 4], :, 4:20] = 0
    c.pos.copy_(good)
    c.run()
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    c.check(wanted)


def test_qk_norm_rope_special_values():
    # zero heads give zeros; a NaN or an infinity stays within its head
    c = QK(4, 2, 1, 64, 32, 32, HALF, torch.bfloat16)
    c.q[0] = 0
    c.q[1, 5], c.q[2, 70] = float("nan"), float("inf")
    c.run()
    q = c.qo.view(4, 2, 64)
    assert bool((q[0] == 0).all()) and bool(q[1, 0].isnan().all()) and bool(q[1, 1].isfinite().all())
    assert bool(q[2, 0].isfinite().all()) and bool(q[2, 1].isnan().any()) and bool(q[3].isfinite().all())
    assert dsa.dsa_device_error() == 0


def test_far_cache_rows():
    # rows past 2^31 elements of the pool
    T, D, bs = 5, 128, 64
    blocks = (1 << 31) // (bs * D) + 3
    kc = torch.zeros(blocks, bs, 1, D, device="cuda", dtype=torch.bfloat16)
    c = QK(T, 2, 1, D, 64, 0, HALF, torch.bfloat16, values=False)
    c.slot = blocks * bs - 1 - 70 * torch.arange(T, device="cuda")
    wanted = c.want()
    c.kc = kc
    c.run()
    (_, _), (k, kp) = wanted
    ref.close(kc.view(-1, 1, D)[c.slot], k, kp, torch.bfloat16, 2.0 ** -20 + 3 * 2.0 ** -24)
    assert int((kc != 0).any(-1).sum()) == T
    assert dsa.dsa_device_error() == 0


def test_rope_calls_on_streams_and_in_a_graph():
    T, H, D, R = 300, 8, 128, 64
    x = torch.randn(T, H, D, device="cuda", generator=gen(9)).bfloat16()
    cs, pos = torch.empty(512, R, device="cuda"), torch.arange(T, device="cuda", dtype=torch.int32)
    y, z = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def chain(st):
        dsa.dsa_rope_table(dsa.make_rope_params(), R, 0, 512, cs, st)
        dsa.dsa_rope(x, H * D, D, pos, cs, 512, R, 0, INTER, False, T, H, D, BF16, y, H * D, D, st)
        dsa.dsa_rope(y, H * D, D, pos, cs, 512, R, 0, INTER, True, T, H, D, BF16, z, H * D, D, st)

    chain(side)
    side.synchronize()
    y1, z1 = y.clone(), z.clone()
    assert float((z1.float() - x.float()).abs().max()) <= 2.0 ** -6 * float(x.abs().max())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(None)
    for _ in range(3):
        for t in (cs, y, z):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y1) and torch.equal(z, z1)
    assert dsa.dsa_device_error() == 0


# ------------------------------------------------------------------ what is copied, and what stays by itself
@pytest.mark.parametrize("layout", [INTER, HALF])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D, R, off, shift", [(64, 64, 0, 0), (128, 64, 64, 0), (96, 24, 12, 0), (64, 32, 3, 0), (33, 10, 7, 0),
                                              (64, 64, 0, 1)])
def test_values_are_copied_whatever_they_hold(D, R, off, shift, dtype, norm, layout):
    # infinities, NaNs and zeros of both signs, in dims that turn in queries and keys and in dims that do not: nothing of
    # a value's neighbours reaches it, and every bit but a NaN's payload is the input's (rounded to bf16)
    c = QK(23, 3, 2, D, R, off, layout, dtype, norm=norm, shift=shift, seed=3)
    pick = torch.randint(0, 24, c.v.shape, device="cuda", generator=gen(4))
    for i, x in enumerate((float("inf"), -float("inf"), float("nan"), -0.0, 0.0)):
        c.v[pick == i] = x
    wanted = c.v.reshape(23, 2, D).bfloat16()
    c.run()
    got = c.vc[c.slot // c.bs, c.slot % c.bs]
    nan = wanted.isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got.view(torch.int16)[~nan], wanted.view(torch.int16)[~nan])
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("layout", [INTER, HALF])
@pytest.mark.parametrize("D, R, off", [(128, 64, 64), (128, 64, 0), (96, 24, 12), (128, 0, 0), (40, 10, 7)])
def test_gains_that_are_no_numbers_stay_in_their_dims(D, R, off, layout):
    clean, c = (QK(7, 2, 2, D, R, off, layout, torch.float32, seed=5) for _ in range(2))
    still = [d for d in range(D) if not off <= d < off + R]
    hit = {still[1]: float("nan"), still[5]: float("inf"), still[-2]: -float("inf")}
    for d, x in hit.items():
        c.gq[d] = c.gk[d] = x
    outs = []
    for x in (clean, c):
        x.run(k_out=torch.empty(7, 2 * D, device="cuda"))
        outs.append((x.qo.view(7, 2, D), x.ko.view(7, 2, D), x.kc[x.slot // x.bs, x.slot % x.bs].float()))
    rest = [d for d in range(D) if d not in hit]
    for a, b in zip(*outs):
        assert torch.equal(a[..., rest], b[..., rest])
        assert not bool(b[..., list(hit)].isfinite().any())
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("layout", [INTER, HALF])
def test_rope_inverse_under_an_amplitude(layout):
    # y = A R x: with the same table the inverse form gives A R^T g, which is the gradient, and A^2 x for y itself
    T, H, D, R, A = 5, 2, 64, 32, 1.25
    cs = torch.empty(16, R, device="cuda")
    dsa.dsa_rope_table(dsa.make_rope_params(amplitude=A), R, 0, 16, cs)
    pos = torch.tensor([0, 3, 15, 1, 8], device="cuda", dtype=torch.int32)
    x, g, y, grad, back = (torch.randn(T, H, D, device="cuda", generator=gen(s)) for s in range(5))
    call = lambda a, b, inv: dsa.dsa_rope(a, H * D, D, pos, cs, 16, R, 16, layout, inv, T, H, D, F32, b, H * D, D)  # noqa: E731
    call(x, y, False)
    call(g, grad, True)
    call(y, back, True)
    leaf = x.double().requires_grad_(True)
    (ref.rotate(leaf, cs[pos.long()], R, 16, layout == HALF)[0] * g.double()).sum().backward()
    _, part = ref.rotate(g.double(), cs[pos.long()], R, 16, layout == HALF, True)
    ref.close(grad, leaf.grad, part, torch.float32, 3 * 2.0 ** -24)
    # twice three roundings of parts no larger than A (|x0| + |x1|), and cos^2 + sin^2 of a table within 2^-22 A
    turned = torch.ones(D, device="cuda", dtype=torch.float64)
    turned[16:48] = A * A
    size = 2 * A * A * float(x.abs().max())
    assert float((back.double() - x.double() * turned).abs().max()) <= (12 * 2.0 ** -24 + 4 * 2.0 ** -22) * size
    assert dsa.dsa_device_error() == 0
