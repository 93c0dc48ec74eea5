"""The calls that prepare a step's inputs on the GPU, against plain 64-bit references
(prepare_ref.py, where the error bounds are derived): slot assignment (whole numbers, equal),
residual + RMS norm + E4M3, the block-scaled E4M3 product, and a run of them into the
indexer's own calls."""
import numpy as np
import pytest

import parity
import pins
import prepare_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from deepseek_v4_sparse_dsa_gb300 import dsa  # noqa: E402
from oracle import dsa_oracle as orc  # noqa: E402

BF16, F32 = dsa.DSA_REAL_BF16, dsa.DSA_REAL_F32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ slot assignment
class Slots:
    """One step's inputs and poisoned outputs on the GPU."""

    def __init__(self, cached, new, bs, max_tokens=None, stride=None, n_free=None, num_blocks=None, seed=0, extra_rows=1):
        rng = np.random.default_rng(seed)
        self.cached, self.new, self.bs = np.asarray(cached, np.int32), np.asarray(new, np.int32), bs
        B = len(self.cached)
        have = -(-self.cached.astype(np.int64) // bs)
        want = -(-(self.cached.astype(np.int64) + np.maximum(self.new, 0)) // bs)
        self.stride = int(max(1, want.max() if B else 1)) if stride is None else stride
        need = int((want - have).sum())
        self.n_free = need if n_free is None else n_free
        pool = rng.permutation(int(have.sum()) + self.n_free + 3).astype(np.int32)
        self.num_blocks = len(pool) if num_blocks is None else num_blocks
        self.table = np.full((B + extra_rows, self.stride), -7, np.int32)
        at = 0
        for b in range(B):
            h = min(int(have[b]), self.stride)
            self.table[b, :h] = pool[at:at + h]
            at += int(have[b])
        self.free = pool[at:at + self.n_free]
        self.tokens = int(np.maximum(self.new, 0).sum()) if max_tokens is None else max_tokens

    def run(self, stream=None):
        B = len(self.cached)
        full = lambda n, t: torch.full((n,), -99, dtype=t, device="cuda")  # noqa: E731
        self.out = dict(table=dev(self.table), ctx=full(B + 1, torch.int32), start=full(B + 2, torch.int32),
                        slot=full(self.tokens + 3, torch.int64), pos=full(self.tokens + 3, torch.int32),
                        used=full(2, torch.int32))
        o = self.out
        self.d = (dev(self.cached), dev(self.new), dev(self.free))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        dsa.dsa_assign_slots(self.d[0], self.d[1], B, self.bs, self.d[2], self.n_free, self.num_blocks, o["table"],
                             self.stride, self.tokens, o["ctx"], o["start"], o["slot"], o["pos"], o["used"], stream)
        err = dsa.dsa_device_error(stream)
        g = {k: v.cpu().numpy() for k, v in o.items()}
        # nothing behind an output's end is touched
        assert g["ctx"][B] == -99 and g["start"][B + 1] == -99 and g["used"][1] == -99
        assert (g["slot"][self.tokens:] == -99).all() and (g["pos"][self.tokens:] == -99).all()
        return err, g["table"], g["ctx"][:B], g["start"][:B + 1], g["slot"][:self.tokens], g["pos"][:self.tokens], int(g["used"][0])

    def check(self, stream=None):
        got = self.run(stream)
        assert got[0] == 0
        want = ref.assign_slots(self.cached, self.new, self.bs, self.free, self.num_blocks, self.table, self.tokens)
        for g, w in zip(got[1:6], want[:5]):
            assert np.array_equal(g, w)
        assert got[6] == want[5]


@pytest.mark.parametrize("cached,new,bs,max_tokens", [
    ([0], [1], 64, None),                               # the first token of the first request
    ([63, 64, 65], [1, 1, 1], 64, None),                # the last slot of a page, a new page, inside a page
    ([5, 0, 9, 3], [0, 0, 0, 0], 4, 5),                 # nothing new
    ([7, 0, 100], [1, 1100, 0], 1, 1200),               # a page per token; a request over two tiles of tokens
    ([0, 1, 1023, 1024, 1025], [1023, 1, 1, 1, 1025], 16, 2100),
    ([130000], [5000], 20, 5003),                       # an odd page size
    ([2**31 - 3], [2], 2**30, None),                    # positions up to INT32_MAX - 1
])
def test_assign_slots(cached, new, bs, max_tokens):
    stride = None if bs < 2**30 else 2
    Slots(cached, new, bs, max_tokens, stride).check()


@pytest.mark.parametrize("B,bs,ctx,most", [(64, 64, 70000, 1), (1000, 16, 3000, 30), (1024, 8, 50, 2), (1025, 128, 500, 9),
                                           (5000, 32, 200, 3)])
def test_assign_slots_batches(B, bs, ctx, most):
    rng = np.random.default_rng(B)
    new = rng.integers(0, most + 1, B)
    Slots(rng.integers(0, ctx, B), new, bs, int(new.sum()) + 7, seed=B).check()
    Slots(rng.integers(0, ctx, B), np.full(B, most), bs, seed=B + 1).check(torch.cuda.Stream())


def test_assign_slots_largest_batch_and_offsets_past_32_bits():
    # 65536 requests with table rows of 40000 entries: 2.6e9 entries, the last rows past 2^31
    B, stride, bs = 65536, 40000, 16
    table = torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
    cached = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    new[0], new[-1], new[-2], cached[-2] = 1, 2, 3, 30
    table[-2, :2] = torch.tensor([3, 4], dtype=torch.int32)
    free = torch.arange(10, 20, dtype=torch.int32, device="cuda")
    ctx, start, used = torch.empty_like(cached), torch.empty(B + 1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    slot, pos = torch.empty(8, dtype=torch.int64, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda")
    dsa.dsa_assign_slots(cached, new, B, bs, free, 10, 100, table, stride, 8, ctx, start, slot, pos, used)
    assert dsa.dsa_device_error() == 0
    assert slot.tolist() == [160, 4 * 16 + 14, 4 * 16 + 15, 11 * 16, 12 * 16, 12 * 16 + 1, -1, -1]
    assert pos.tolist() == [0, 30, 31, 32, 0, 1, 0, 0] and int(used) == 3
    assert table[-2, :4].tolist() == [3, 4, 11, -1] and table[-1, :2].tolist() == [12, -1] and int(table[0, 0]) == 10
    assert int((table != -1).sum()) == 5
    assert start[:3].tolist() == [0, 1, 1] and start[-3:].tolist() == [1, 4, 6] and torch.equal(ctx, cached + new)


def test_assign_slots_no_requests():
    err, table, ctx, start, slot, pos, used = Slots([], [], 64, 9, 1).run()
    assert err == 0 and start.tolist() == [0] and used == 0
    assert (slot == -1).all() and (pos == 0).all() and (table == -7).all()


def test_assign_slots_flags_what_does_not_fit():
    I = dsa.DSA_DEVERR_INDEX
    # a free list of exactly the pages needed (one for the first request, two for the second)
    s = Slots([0, 3], [4, 9], 4, n_free=3)
    err, table, ctx, start, slot, pos, used = s.run()
    assert err == 0 and used == 3
    # one page short: the last page's tokens have no slot, its entry is -1, the need is reported
    s = Slots([0, 3], [4, 9], 4, n_free=2)
    err, table, ctx, start, slot, pos, used = s.run()
    assert err == I and used == 3 and ctx.tolist() == [4, 12]
    assert table[1].tolist()[1:] == [s.free[1], -1]
    assert (slot[-4:] == -1).all() and (slot[:-4] >= 0).all() and pos[-4:].tolist() == [8, 9, 10, 11]
    # a table row too short
    err, table, ctx, start, slot, pos, used = Slots([2, 0], [4, 1], 2, stride=2).run()
    assert err == I and slot[:2].min() >= 0 and (slot[2:4] == -1).all() and slot[4] >= 0
    # block ids outside the pool: one held, one from the free list
    s = Slots([3, 0], [1, 1], 4)
    s.table[0, 0], s.free[0] = s.num_blocks, -5
    err, table, ctx, start, slot, pos, used = s.run()
    assert err == I and slot.tolist() == [-1, -1] and table[1, 0] == -1 and table[0, 0] == s.num_blocks
    # more tokens than max_tokens: those past it get neither slot nor page
    s = Slots([0, 0], [3, 6], 4, max_tokens=5)
    err, table, ctx, start, slot, pos, used = s.run()
    assert err == I and start.tolist() == [0, 3, 9] and used == 3 and (slot >= 0).all()
    assert table[1].tolist() == [s.free[1], -7]
    # negative lengths and sums past 32 bits: such a request brings nothing, the others keep theirs
    s = Slots([5, 4, 2**31 - 1, 0], [1, 1, 1, 2], 4, stride=4, max_tokens=4)
    s.cached[0], s.new[1] = -1, -3
    err, table, ctx, start, slot, pos, used = s.run()
    assert err == I and ctx.tolist() == [0, 4, 2**31 - 1, 2] and start.tolist() == [0, 0, 0, 0, 2]
    assert (slot[:2] >= 0).all() and (slot[2:] == -1).all() and used == 1


# ------------------------------------------------------------------ norm
def norm_case(T, D, typ, residual=True, want_y=True, want_codes=True, pow2=False, pad=0, seed=0, x=None, scale_x=1.0,
              stream=None):
    rng = np.random.default_rng(seed + 31 * T + D)
    tt = torch.bfloat16 if typ == BF16 else torch.float32
    g = dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    mk = lambda: dev((rng.standard_normal((T, D + pad)) * scale_x).astype(np.float32)).to(tt)  # noqa: E731
    x = mk() if x is None else x
    res = mk() if residual else None
    ld = D + pad
    ro = torch.full((T, ld), 7.0, dtype=tt, device="cuda") if residual else None
    y = torch.full((T, ld), 7.0, dtype=tt, device="cuda") if want_y else None
    codes = torch.full((T, ld), 0x5A, dtype=torch.uint8, device="cuda") if want_codes else None
    scale = torch.full((T, -(-D // 128)), float("nan"), device="cuda") if want_codes else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    dsa.dsa_add_rmsnorm_e4m3(x, ld, res, ld, g, 1e-6, T, D, typ, ro, y, codes, ld, scale, pow2, stream)
    assert dsa.dsa_device_error(stream) == 0
    r64, y64 = ref.add_rmsnorm(f64(x)[:, :D], None if res is None else f64(res)[:, :D], f64(g), float(np.float32(1e-6)), typ == BF16)
    if ro is not None:
        assert np.array_equal(f64(ro)[:, :D], r64)
        assert (f64(ro)[:, D:] == 7.0).all()
    if y is not None:
        half = 2.0 ** -8 if typ == BF16 else 2.0 ** -24
        assert (np.abs(f64(y)[:, :D] - y64) <= (ref.Y_REL + half + ref.Y_REL * half) * np.abs(y64) + 2.0 ** -133).all()
        assert (f64(y)[:, D:] == 7.0).all()
    if codes is not None:
        c = codes.cpu().numpy()
        ref.check_quantised(y64, c[:, :D], scale.cpu().numpy(), pow2)
        assert (c[:, D:] == 0x5A).all()


@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (2, 127), (5, 128), (4, 129), (33, 1000), (7, 1536), (1, 4096), (9, 4100),
                                 (3, 5001), (2, 8192), (2, 8200), (2, 9000), (1, 16384), (2, 20011), (1, 32768), (700, 512)])
def test_add_rmsnorm(T, D, typ):
    norm_case(T, D, typ)


@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("D", [4104, 6143, 6144, 6145, 6152, 8185, 8192])
@pytest.mark.parametrize("rows", [(0, 31), (1, 0), (1, 1), (2, 0), (2, 1)])
def test_add_rmsnorm_wide_rows(rows, D, typ):
    # a row per SM, two, and one more: where a thread's share of a row changes
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    norm_case(rows[0] * sms + rows[1], D, typ)


@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("D", [8193, 8200, 16383, 16384, 16385])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_add_rmsnorm_widest_rows(more, D, typ):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    norm_case(sms + more, D, typ, residual=more < 1)


def test_add_rmsnorm_wide_rows_past_the_cache():
    # rows of 12288 that exceed 96 MiB, every output: the last rows, and rows of a small batch, agree with the formula
    T, D = 1000, 12288
    x, res = torch.randn(T, D, device="cuda").to(torch.bfloat16), torch.randn(T, D, device="cuda").to(torch.bfloat16)
    g = torch.rand(D, device="cuda") + 0.5
    ro, y = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 128, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, D, res, D, g, 1e-6, T, D, BF16, ro, y, codes, D, scale)
    at = np.r_[0:8, 148:156, 300:308, T - 8:T]
    r64, y64 = ref.add_rmsnorm(f64(x[at]), f64(res[at]), f64(g), float(np.float32(1e-6)), True)
    assert np.array_equal(f64(ro[at]), r64)
    half = 2.0 ** -8
    assert (np.abs(f64(y[at]) - y64) <= (ref.Y_REL + half + ref.Y_REL * half) * np.abs(y64) + 2.0 ** -133).all()
    ref.check_quantised(y64, codes[at].cpu().numpy(), scale[at].cpu().numpy(), False)
    assert torch.equal(ro, (x.float() + res.float()).to(torch.bfloat16))


@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(residual=False), dict(want_y=False), dict(want_codes=False), dict(pow2=True),
                                dict(pad=1), dict(pad=8, pow2=True), dict(pad=4), dict(scale_x=1e-3), dict(scale_x=100.0)])
def test_add_rmsnorm_options(typ, kw):
    for D in (264, 3000, 9000):
        norm_case(6, D, typ, **kw)


def test_add_rmsnorm_misaligned_and_other_stream():
    base = torch.randn(5, 300, device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()
    norm_case(5, 256, BF16, x=base[:, 1:257].contiguous(), residual=False, stream=s)
    # rows that start 2 bytes off a 16-byte boundary
    x = torch.randn(4 * 256 + 8, device="cuda").to(torch.bfloat16)
    g = torch.ones(256, device="cuda")
    for off in (0, 1, 4):
        v = x[off:off + 1024].view(4, 256)
        codes = torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
        scale = torch.zeros(4, 2, device="cuda")
        dsa.dsa_add_rmsnorm_e4m3(v, 256, None, 0, g, 1e-6, 4, 256, BF16, None, None, codes, 256, scale)
        _, y64 = ref.add_rmsnorm(f64(v), None, f64(g), float(np.float32(1e-6)), True)
        ref.check_quantised(y64, codes.cpu().numpy(), scale.cpu().numpy(), False)


def test_add_rmsnorm_in_place():
    # the residual stream updated in place, and y written over x, equal the separate buffers
    for typ, tt in ((BF16, torch.bfloat16), (F32, torch.float32)):
        for D in (640, 4096, 4099):
            x, res = torch.randn(37, D, device="cuda").to(tt), torch.randn(37, D, device="cuda").to(tt)
            g = torch.rand(D, device="cuda") + 0.5
            ro, y = torch.empty_like(x), torch.empty_like(x)
            dsa.dsa_add_rmsnorm_e4m3(x, D, res, D, g, 1e-5, 37, D, typ, ro, y, None, D, None)
            x2, res2 = x.clone(), res.clone()
            dsa.dsa_add_rmsnorm_e4m3(x2, D, res2, D, g, 1e-5, 37, D, typ, res2, x2, None, D, None)
            assert torch.equal(res2, ro) and torch.equal(x2, y)
            x3 = x.clone()
            dsa.dsa_add_rmsnorm_e4m3(x3, D, res, D, g, 1e-5, 37, D, typ, x3, None, None, D, None)
            assert torch.equal(x3, ro)


def test_add_rmsnorm_zero_rows_and_non_finite():
    x = torch.zeros(4, 256, device="cuda")
    x[1, 5] = 3.0
    x[2, 7] = float("nan")
    x[3, 200] = float("inf")
    g = torch.ones(256, device="cuda")
    codes = torch.full((4, 256), 0x11, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(4, 2, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, 256, None, 0, g, 1e-6, 4, 256, F32, None, None, codes, 256, scale)
    c, s = codes.cpu().numpy(), scale.cpu().numpy()
    assert (c[0] == 0).all() and (s[0] == 1).all()                  # an all-zero row
    assert c[1, 5] == 0x7E and (np.delete(c[1], 5) == 0).all() and s[1, 1] == 1   # one live element, a zero group
    assert ((c[2] & 0x7F) == 0x7F).all()                            # NaN row
    assert (c[3, 200] & 0x7F) == 0x7F and (np.delete(c[3], 200) & 0x7F == 0).all()


def test_add_rmsnorm_bf16_subnormals_and_offsets_past_32_bits():
    # sums of bf16 subnormals are exact and kept
    x = torch.full((2, 256), 9.2e-41, device="cuda").to(torch.bfloat16)
    res = torch.full((2, 256), 1.8e-40, device="cuda").to(torch.bfloat16)
    assert x[0, 0] > 0 and res[0, 0] > 0
    ro, g = torch.empty_like(x), torch.ones(256, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, 256, res, 256, g, 1e-6, 2, 256, BF16, ro, None, None, 0, None)
    assert np.array_equal(f64(ro), f64(x) + f64(res))
    # 2.3e9 elements: the last rows against the same rows alone
    T, D = 70000, 32768
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[-40:] = torch.randn(40, D, device="cuda").to(torch.bfloat16)
    g = torch.rand(D, device="cuda") + 0.5
    codes, scale = torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 128, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, D, None, 0, g, 1e-6, T, D, BF16, None, None, codes, D, scale)
    assert dsa.dsa_device_error() == 0
    _, y64 = ref.add_rmsnorm(f64(x[-40:]), None, f64(g), float(np.float32(1e-6)), True)
    ref.check_quantised(y64, codes[-40:].cpu().numpy(), scale[-40:].cpu().numpy(), False)
    assert not codes[:-40].any() and bool((scale[:-40] == 1).all())


def test_add_rmsnorm_rows_do_not_depend_on_the_batch():
    x = torch.randn(300, 1536, device="cuda").to(torch.bfloat16)
    g = torch.rand(1536, device="cuda")

    def call(v):
        c = torch.empty(v.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(v.shape[0], 12, device="cuda")
        dsa.dsa_add_rmsnorm_e4m3(v, 1536, None, 0, g, 1e-6, v.shape[0], 1536, BF16, None, None, c, 1536, s)
        return c, s
    c, s = call(x)
    c1, s1 = call(x[17:18])
    assert torch.equal(c[17:18], c1) and torch.equal(s[17:18], s1)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("D", [384, 381])
def test_add_rmsnorm_tiny_groups(D, typ, pow2):
    # a group of tiny values with zeros among them, down to subnormals, in an otherwise zero row and beside a
    # normal group: neither 1 / scale nor 1 / rms times it may overflow.  Powers of two for gamma: r gamma is exact.
    tiny = [1e-29, 1e-32, 1e-35, 1.2e-36, 1e-36, 3e-37, 1e-38, 1e-39, 9.2e-41]
    T = 2 * len(tiny)
    x = torch.zeros(T, D)
    part = torch.tensor([1.0, 0.5, 0.0, -0.25, -1.0, 0.3, 0.0, 0.001])
    for i, t in enumerate(tiny):
        x[2 * i:2 * i + 2, 40:48] = t * part
        x[2 * i + 1, 256:] = torch.randn(D - 256)
    x = x.cuda().to(torch.bfloat16 if typ == BF16 else torch.float32)
    g = torch.tensor([1.0, 2.0], device="cuda").repeat(D)[:D].contiguous()
    codes = torch.full((T, D), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((T, 3), float("nan"), device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, D, None, 0, g, 1e-6, T, D, typ, None, None, codes, D, scale, pow2)
    _, y64 = ref.add_rmsnorm(f64(x), None, f64(g), float(np.float32(1e-6)), typ == BF16)
    ref.check_quantised(y64, codes.cpu().numpy(), scale.cpu().numpy(), pow2)


def test_add_rmsnorm_tiny_group_by_hand():
    # 1 / rms is 1000, max|y| = 1.2e-33: the largest value is 448 times its scale, half of it 224, zeros stay zero
    x = torch.zeros(1, 128, device="cuda")
    x[0, 0], x[0, 1] = 1.2e-36, 6e-37
    codes, scale = torch.zeros(1, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, 128, None, 0, torch.ones(128, device="cuda"), 1e-6, 1, 128, F32, None, None, codes, 128, scale)
    assert codes[0, :3].tolist() == [0x7E, 0x76, 0] and not codes[0, 2:].any()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("typ", [BF16, F32])
@pytest.mark.parametrize("D", [384, 381])
def test_add_rmsnorm_scales_of_non_finite_rows(D, typ, pow2):
    # the codes tell: NaN everywhere in a row that holds a NaN; NaN at an infinity's place and zeros elsewhere.  Every
    # scale of such a row is 1, so that what is finite stays finite when the codes are multiplied by it
    x = torch.randn(4, D, device="cuda")
    x[0, 200], x[1, 5], x[2, 300] = float("inf"), float("nan"), float("-inf")
    x = x.to(torch.bfloat16 if typ == BF16 else torch.float32)
    codes, scale = torch.zeros(4, D, dtype=torch.uint8, device="cuda"), torch.zeros(4, 3, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, D, None, 0, torch.ones(D, device="cuda"), 1e-6, 4, D, typ, None, None, codes, D, scale, pow2)
    c = codes.cpu().numpy() & 0x7F
    assert bool((scale[:3] == 1.0).all()) and bool(torch.isfinite(scale[3]).all())
    assert (c[1] == 0x7F).all()
    for row, at in ((0, 200), (2, 300)):
        assert c[row, at] == 0x7F and (np.delete(c[row], at) == 0).all()
    _, y64 = ref.add_rmsnorm(f64(x[3:]), None, np.ones(D), float(np.float32(1e-6)), typ == BF16)
    ref.check_quantised(y64, codes[3:].cpu().numpy(), scale[3:].cpu().numpy(), pow2)


def test_add_rmsnorm_rows_of_batches_on_both_sides_of_the_thread_split():
    # up to two rows per SM a row takes twice the threads: within one launch shape a row's bits do not depend on its
    # neighbours; across the limit its sum of squares has another order, and both results hold against 64 bits
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    x = torch.randn(n + 1, 1536, device="cuda").to(torch.bfloat16)
    g = torch.rand(1536, device="cuda") + 0.5
    _, y64 = ref.add_rmsnorm(f64(x), None, f64(g), float(np.float32(1e-6)), True)

    def call(v):
        c = torch.empty(v.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(v.shape[0], 12, device="cuda")
        dsa.dsa_add_rmsnorm_e4m3(v, 1536, None, 0, g, 1e-6, v.shape[0], 1536, BF16, None, None, c, 1536, s)
        return c, s
    few, many, more = call(x[:n]), call(x), call(torch.cat((x, x)))
    for c, s in (few, many, more):
        m = min(len(c), n + 1)
        ref.check_quantised(y64[:m], c[:m].cpu().numpy(), s[:m].cpu().numpy(), False)
    assert all(torch.equal(p, q[:n + 1]) and torch.equal(p, q[n + 1:]) for p, q in zip(many, more))
    for rows in (slice(17, 18), slice(0, 40), slice(n - 1, n)):
        assert all(torch.equal(p[rows], q) for p, q in zip(few, call(x[rows])))


@pytest.mark.parametrize("typ", [BF16, F32])
def test_add_rmsnorm_power_of_two_scales_of_a_prompt(typ):
    # The scale before it is rounded up: |r gamma| and the two products round at 2^-24 each, 1 / 448 is off by at most that;
    # 1 / rms by the root's 2 ulps (2^-22) and half the sum of squares' error, a thread's 16 squares, 5 + 8 sums of warps
    # and the mean: 31 roundings of 2^-24.  Together 23.5 * 2^-24 < 2^-19: farther than that from a power of two the
    # exponent is the 64-bit one, nearer it is that or its neighbour.
    T, D = 16384, 4096
    tt = torch.bfloat16 if typ == BF16 else torch.float32
    x = torch.randn(T, D, device="cuda").to(tt)
    g = torch.rand(D, device="cuda") + 0.5
    codes, scale = torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 128, device="cuda")
    dsa.dsa_add_rmsnorm_e4m3(x, D, None, 0, g, 1e-6, T, D, typ, None, None, codes, D, scale, True)
    near = 0
    for t in range(0, T, 2048):
        r = x[t:t + 2048].double()
        y = r / (r.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt() * g.double()
        want = torch.log2(y.view(2048, D // 128, 128).abs().amax(-1) / 448.0)
        m, e = torch.frexp(scale[t:t + 2048])
        assert bool((m == 0.5).all())
        got = (e - 1).double()
        edge = (want - want.round()).abs() < 1.5 * 2.0 ** -19       # log2(1 + d) < 1.5 d
        near += int(edge.sum())
        assert bool((got == want.ceil())[~edge].all())
        assert bool(((got - want.round()) * (got - want.round() - 1) == 0)[edge].all())
        q = codes[t:t + 2048].view(torch.float8_e4m3fn).double() * scale[t:t + 2048].double().repeat_interleave(128, 1)
        # half a code's step, 2^-4 relative, and y's own error (at most 2^-18)
        assert bool(((q - y).abs() <= (2.0 ** -4 + 2.0 ** -17) * y.abs() + scale[t:t + 2048].double().repeat_interleave(128, 1) * 2.0 ** -10).all())
    assert near < 20                                      # of 524288 groups some 4 x 2^-19 of them are expected there


def test_add_rmsnorm_power_of_two_scales_at_the_border():
    # mean(r^2) + eps = 4: y = r gamma / 2, and a largest value of 448 2^k gives a scale of 2^k.  2^-18 above it the next
    # power, 2^-18 below it the same; on the border itself the root's last bit decides between the two
    x = torch.ones(6, 256, device="cuda").to(torch.bfloat16)
    for k in (-3, 0, 5):
        for d, want in ((0.0, (1, 2)), (2.0 ** -18, (2,)), (-2.0 ** -18, (1,))):
            g = torch.full((256,), 0.25, device="cuda")
            g[7], g[200] = 896.0 * 2.0 ** k * (1 + d), -896.0 * 2.0 ** k * (1 + d)
            codes, scale = torch.empty(6, 256, dtype=torch.uint8, device="cuda"), torch.empty(6, 2, device="cuda")
            dsa.dsa_add_rmsnorm_e4m3(x, 256, None, 0, g, 3.0, 6, 256, BF16, None, None, codes, 256, scale, True)
            assert set((scale / 2.0 ** k).flatten().tolist()) <= {float(w) for w in want}
            top = codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, 1)
            assert bool(((top[:, 7] - 448.0 * 2.0 ** k).abs() <= 448.0 * 2.0 ** k * 2.0 ** -17).all())


# ------------------------------------------------------------------ gemm
def gemm_inputs(M, N, K, seed=0, lda=None, ldw=None, signed=False, codes=None):
    rng = np.random.default_rng(seed + M + 7 * N + 13 * K)
    lda, ldw = lda or -(-K // 16) * 16, ldw or -(-K // 16) * 16
    # codes of quantised normals: all magnitudes below NaN, weighted to the upper exponents
    draw = lambda r, ld: np.where(rng.random((r, ld)) < 0.5, rng.integers(0x30, 0x7F, (r, ld)),  # noqa: E731
                                  rng.integers(0, 0x7F, (r, ld))).astype(np.uint8) | (rng.integers(0, 2, (r, ld)) << 7).astype(np.uint8)
    a, w = draw(M, lda), draw(N, ldw)
    a[:, K:], w[:, K:] = 0x7F, 0x7F                     # NaN past K: not part of the product
    G = -(-K // 128)
    sgn = (lambda s: np.where(rng.random(s) < 0.3, -1, 1)) if signed else (lambda s: 1)
    asc = ((0.1 + rng.random((M, G))) * sgn((M, G))).astype(np.float32)
    wsc = ((0.1 + rng.random((-(-N // 128), G))) * 1e-3 * sgn((-(-N // 128), G))).astype(np.float32)
    return a, asc, w, wsc


def gemm_call(a, asc, w, wsc, K, typ, ldo=None, stream=None):
    M, N = a.shape[0], w.shape[0]
    ldo = ldo or N
    out = torch.full((M, ldo), 7.0, dtype=torch.bfloat16 if typ == BF16 else torch.float32, device="cuda")
    d = [dev(v) for v in (a, asc, w, wsc)]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    dsa.dsa_gemm_e4m3(d[0], a.shape[1], d[1], d[2], w.shape[1], d[3], M, N, K, out, ldo, typ, stream)
    assert dsa.dsa_device_error(stream) == 0
    return out


def gemm_check(M, N, K, typ, ldo=None, **kw):
    a, asc, w, wsc = gemm_inputs(M, N, K, **kw)
    out = f64(gemm_call(a, asc, w, wsc, K, typ, ldo))
    want, tol = ref.gemm(a[:, :K], asc, w[:, :K], wsc)
    if typ == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(out[:, :N] - want)
    assert (err <= tol).all(), (err / tol).max()
    assert (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(128, 128), (64, 512), (200, 1000), (1000, 2064)])
def test_gemm(M, N, K):
    gemm_check(M, N, K, F32)
    gemm_check(M, N, K, BF16, seed=1)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 17), (1, 8192, 2048), (5, 129, 127), (40, 1, 4096), (2, 130, 16384),
                                   (1000, 64, 640), (513, 700, 384), (2048, 2048, 256), (600, 1300, 1408)])
def test_gemm_sizes(M, N, K):
    gemm_check(M, N, K, F32)


@pytest.mark.parametrize("M", [7, 100, 700])
def test_gemm_strides_and_signed_scales(M):
    gemm_check(M, 333, 650, BF16, ldo=340, lda=672, ldw=704, signed=True)
    gemm_check(M, 333, 650, F32, ldo=335, lda=656, ldw=1024, signed=True)


def test_gemm_large_product():
    # more tiles than the GPU holds at once; checked on sampled rows
    M, N, K = 4099, 4100, 1024
    a, asc, w, wsc = gemm_inputs(M, N, K)
    out = gemm_call(a, asc, w, wsc, K, BF16)
    rows = np.r_[0:3, 127:130, 2047:2050, M - 130:M]
    want, tol = ref.gemm(a[rows], asc[rows], w, wsc)
    assert (np.abs(f64(out)[rows] - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
    # the same call twice: the same bits
    assert torch.equal(out, gemm_call(a, asc, w, wsc, K, BF16))


@pytest.mark.parametrize("M,N,K,ldo", [(2000, 2304, 384, 2304), (2304, 2000, 1000, 2008), (1500, 2600, 4112, 2601),
                                       (129, 19500, 160, 19500), (19500, 129, 160, 136)])
@pytest.mark.parametrize("typ", [BF16, F32])
def test_gemm_many_tiles(M, N, K, ldo, typ):
    # whole and ragged tiles in both directions, K past its last whole block, stores of 16 bytes and less
    gemm_check(M, N, K, typ, ldo=ldo, signed=True)


@pytest.mark.parametrize("M,N,K", [(1, 19456, 160), (1, 19457, 160), (16, 24576, 144), (17, 24577, 144), (64, 32768, 128),
                                   (128, 19456, 128), (130, 9800, 272), (200, 9856, 256), (256, 9984, 256), (257, 6500, 400)])
@pytest.mark.parametrize("typ", [BF16, F32])
def test_gemm_few_tokens_with_many_columns(M, N, K, typ):
    # on both sides of the number of tiles that sends a product to the CTA pairs, down to one token
    gemm_check(M, N, K, typ, signed=True)


def test_gemm_offsets_past_32_bits():
    # rows 1 MiB apart: the last rows of a and out lie past 4 GiB and 2^32 elements
    M, N, K, ld = 4500, 128, 256, 1 << 20
    a, asc, w, wsc = gemm_inputs(M, N, K)
    want = gemm_call(a, asc, w, wsc, K, BF16)
    big = torch.zeros(M, ld, dtype=torch.uint8, device="cuda")
    big[:, :K] = dev(a)
    out = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
    d = [dev(v) for v in (asc, w, wsc)]
    dsa.dsa_gemm_e4m3(big, ld, d[0], d[1], K, d[2], M, N, K, out, ld, BF16)
    assert dsa.dsa_device_error() == 0
    assert torch.equal(out[:, :N], want) and not out[:, N:].any()


def test_gemm_one_row_of_any_stride():
    # one row's stride is never used: out rows may be any distance apart, also where it exceeds 2^40 bytes
    a, asc, w, wsc = gemm_inputs(1, 19600, 256)
    want, tol = ref.gemm(a, asc, w, wsc)
    d = [dev(v) for v in (a, asc, w, wsc)]
    for typ, tt in ((F32, torch.float32), (BF16, torch.bfloat16)):
        for ldo in (1 << 40, 1 << 61, 1 << 62):
            out = torch.full((1, 19600), 7.0, dtype=tt, device="cuda")
            dsa.dsa_gemm_e4m3(d[0], 256, d[1], d[2], 256, d[3], 1, 19600, 256, out, ldo, typ)
            assert dsa.dsa_device_error() == 0
            half = 2.0 ** -8 if typ == BF16 else 0.0
            assert (np.abs(f64(out) - want) <= tol + half * (np.abs(want) + tol)).all()


def test_gemm_on_two_streams_at_once():
    # products of different shapes in flight together, each repeated: every result as when run alone
    cases = [(gemm_inputs(m, n, k), k) for m, n, k in ((3, 700, 2048), (300, 900, 1024), (2300, 2100, 512))]
    want = [gemm_call(*c, k, BF16) for c, k in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    data = [[dev(v) for v in c] for c, _ in cases]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    torch.cuda.synchronize()
    for i in range(10):
        for (a, asc, w, wsc), (_, k), st, o in zip(data, cases, streams, outs):
            dsa.dsa_gemm_e4m3(a, a.shape[1], asc, w, w.shape[1], wsc, a.shape[0], w.shape[0], k, o[i], w.shape[0], BF16, st)
    for st in streams:
        assert dsa.dsa_device_error(st) == 0
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_gemm_non_finite_stays_in_its_row_and_column():
    a, asc, w, wsc = gemm_inputs(40, 200, 512)
    a[3, 100] = 0x7F
    asc[5, 1] = np.inf
    w[7, 200] = 0xFF
    out = f64(gemm_call(a, asc, w, wsc, 512, F32))
    bad = ~np.isfinite(out)
    assert bad[3].all() and bad[5].all() and bad[:, 7].all()
    bad[[3, 5]], bad[:, 7] = False, False
    assert not bad.any()


def test_gemm_other_stream_and_graph():
    a, asc, w, wsc = gemm_inputs(20, 500, 1024)
    K = 1024
    want = gemm_call(a, asc, w, wsc, K, F32)
    assert torch.equal(want, gemm_call(a, asc, w, wsc, K, F32, stream=torch.cuda.Stream()))
    d = [dev(v) for v in (a, asc, w, wsc)]
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_gemm_e4m3(d[0], K, d[1], d[2], K, d[3], 20, 500, K, out, 500, F32)
    for seed in (5, 6):
        a2, asc2, _, _ = gemm_inputs(20, 500, 1024, seed=seed)
        d[0].copy_(dev(a2))
        d[1].copy_(dev(asc2))
        out.zero_()
        graph.replay()
        assert torch.equal(out, gemm_call(a2, asc2, w, wsc, K, F32))


@pytest.mark.parametrize("M,N", [(5, 300), (100, 900), (2100, 2300)])
def test_calls_behind_copies_and_other_kernels_in_a_graph(M, N):
    # a captured chain copy -> norm -> product -> norm of the product: each starts early behind a kernel, and
    # whole behind a copy; replayed on new inputs it gives what the eager calls give
    K = 512
    a, asc, w, wsc = gemm_inputs(8, N, K)
    dw, dws, g, g2 = dev(w), dev(wsc), torch.rand(K, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    src, x = e(M, K, t=torch.bfloat16), e(M, K, t=torch.bfloat16)
    codes, scale, out, y = e(M, K, t=torch.uint8), e(M, K // 128), e(M, N), e(M, N)

    def chain():
        x.copy_(src)
        dsa.dsa_add_rmsnorm_e4m3(x, K, None, 0, g, 1e-6, M, K, BF16, None, None, codes, K, scale)
        dsa.dsa_gemm_e4m3(codes, K, scale, dw, K, dws, M, N, K, out, N, F32)
        dsa.dsa_add_rmsnorm_e4m3(out, N, None, 0, g2, 1e-6, M, N, F32, None, y, None, N, None)
        dsa.dsa_gemm_e4m3(codes, K, scale, dw, K, dws, M, N, K, out, N, F32)
    src.normal_()
    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            chain()
    for _ in range(4):
        src.normal_()
        chain()
        want = (codes.clone(), scale.clone(), out.clone(), y.clone())
        for t in (codes, scale, out, y):
            t.zero_()
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(want, (codes, scale, out, y)))
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("M", [5, 24, 100, 2100])
def test_a_chain_whose_scales_change_from_link_to_link(M):
    # product -> norm -> product over the same code and scale buffers, nothing between them: a product is resident
    # before the norm in front of it has written its scales, while the product before that still reads the old ones
    D, links = 2304, 6
    a, asc, w, wsc = gemm_inputs(M, D, D)
    dw, dws = dev(w), dev(wsc)
    gammas = [torch.rand(D, device="cuda") * 2.0 ** (3 * i % 8) + 0.1 for i in range(links)]
    start = torch.randn(M, D, device="cuda")
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    codes, scale, out = e(M, D, t=torch.uint8), e(M, D // 128), e(M, D)
    seen = [(torch.empty_like(codes), torch.empty_like(scale), torch.empty_like(out)) for _ in range(links)]

    def chain(apart):
        src = start
        for i, g in enumerate(gammas):
            dsa.dsa_add_rmsnorm_e4m3(src, D, None, 0, g, 1e-6, M, D, F32, None, None, codes, D, scale)
            if apart:
                torch.cuda.synchronize()
            dsa.dsa_gemm_e4m3(codes, D, scale, dw, D, dws, M, D, D, out, D, F32)
            if apart:
                torch.cuda.synchronize()
                for t, s in zip((codes, scale, out), seen[i]):
                    s.copy_(t)
            src = out

    chain(True)
    assert all(not torch.equal(seen[i][1], seen[i + 1][1]) for i in range(links - 1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            chain(False)
    for _ in range(10):
        for t in (codes, scale, out):
            t.zero_()
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip((codes, scale, out), seen[-1]))
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("T", [3, 70])
def test_a_product_feeds_the_sparse_attention(T):
    # product -> attention over one query buffer, whose rows change from link to link: the attention is resident while
    # the product writes its queries
    from deepseek_v4_sparse_dsa_gb300 import synth
    ab = synth.make_attn(5, [200] * T, 1, 64)
    K, N, links = 512, 64 * 128, 4
    w, wsc = gemm_inputs(8, N, K)[2:]
    d = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    dw, dws, sel, fp4, sc, tab, sink = map(d, (w, wsc, ab.sel, ab.kv_fp4, ab.kv_scale, ab.table, ab.sink))
    acts = [tuple(map(d, gemm_inputs(T, 8, K, seed=i)[:2])) for i in range(links)]
    q, out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), torch.empty(links, T, 64, 128, device="cuda")

    def chain(apart):
        for i, (a, asc) in enumerate(acts):
            dsa.dsa_gemm_e4m3(a, K, asc, dw, K, dws, T, N, K, q, N, BF16)
            if apart:
                torch.cuda.synchronize()
            dsa.dsa_sparse_attn_mxfp4(q, T, 64, 128, sel, ab.topk, fp4, sc, fp4.shape[0], ab.block_size, tab, tab.shape[1],
                                      1, sink, 1e-3, out[i])
            if apart:
                torch.cuda.synchronize()

    chain(True)
    want = out.clone()
    assert all(not torch.equal(want[i], want[i + 1]) for i in range(links - 1)) and bool(torch.isfinite(want).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            chain(False)
    for _ in range(10):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert dsa.dsa_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(4, 256, 4096), (200, 300, 2048), (2000, 2000, 1024)])
def test_gemm_expired_waits_flag_timeout(M, N, K):
    a, asc, w, wsc = gemm_inputs(M, N, K)
    d = [dev(v) for v in (a, asc, w, wsc)]
    out = torch.empty(M, N, device="cuda")
    call = lambda: dsa.dsa_gemm_e4m3(d[0], K, d[1], d[2], K, d[3], M, N, K, out, N, F32)  # noqa: E731
    assert dsa.dsa_device_error() == 0
    dsa.dsa_set_wait_limit_ns(1)
    try:
        call()
        err = dsa.dsa_device_error()
    finally:
        dsa.dsa_set_wait_limit_ns(0)
    assert err >= 0 and err & dsa.DSA_DEVERR_TIMEOUT
    call()
    assert dsa.dsa_device_error() == 0
    want, tol = ref.gemm(a[:8], asc[:8], w, wsc)
    assert (np.abs(f64(out)[:8] - want) <= tol).all()


@pytest.mark.parametrize("out_typ", [BF16, F32])
def test_gemm_pairs_abandoned_again_and_again(out_typ):
    # a pair's CTAs give up at different points: what one still signals to the other arrives before it has left, the
    # context stays usable and the next call is right.  One tile of a pair, and more tiles than pairs.
    for M, N, K in ((300, 9800, 512), (2600, 2600, 640)):
        a, asc, w, wsc = gemm_inputs(M, N, K)
        d = [dev(v) for v in (a, asc, w, wsc)]
        out = torch.empty(M, N, dtype=torch.bfloat16 if out_typ == BF16 else torch.float32, device="cuda")
        call = lambda: dsa.dsa_gemm_e4m3(d[0], K, d[1], d[2], K, d[3], M, N, K, out, N, out_typ)  # noqa: E731
        call()
        want = out.clone()
        assert dsa.dsa_device_error() == 0
        for limit in (1, 500, 2000, 4000, 1):
            dsa.dsa_set_wait_limit_ns(limit)
            try:
                for _ in range(10):
                    call()
                err = dsa.dsa_device_error()
            finally:
                dsa.dsa_set_wait_limit_ns(0)
            assert err >= 0 and err & ~dsa.DSA_DEVERR_TIMEOUT == 0
            out.zero_()
            call()
            assert dsa.dsa_device_error() == 0 and torch.equal(out, want)


SECOND_CONTEXT = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
import torch
from deepseek_v4_sparse_dsa_gb300 import dsa
cu, lib = ctypes.CDLL("libcuda.so.1"), dsa.load()
torch.zeros(1, device="cuda")

def ck(r):
    assert r == 0, r

def products():
    # all ones, all scales one: every output is K
    for M, N, K in ((2000, 2000, 256), (200, 300, 2048), (20, 128, 4096), (3, 128, 4096)):
        g = K // 128
        sizes, p = (M * K, M * g * 4, N * K, -(-N // 128) * g * 4, M * N * 4), []
        for n in sizes:
            p.append(ctypes.c_uint64())
            ck(cu.cuMemAlloc_v2(ctypes.byref(p[-1]), ctypes.c_size_t(n)))
        for i in (0, 2):
            ck(cu.cuMemsetD8_v2(p[i], 0x38, ctypes.c_size_t(sizes[i])))
        for i in (1, 3):
            ck(cu.cuMemsetD32_v2(p[i], 0x3F800000, ctypes.c_size_t(sizes[i] // 4)))
        a, sa, w, sw, o = (v.value for v in p)
        assert lib.dsa_gemm_e4m3(a, K, sa, w, K, sw, M, N, K, o, N, dsa.DSA_REAL_F32, None) == dsa.DSA_OK
        assert lib.dsa_device_error(None) == 0
        host = (ctypes.c_float * (M * N))()
        ck(cu.cuMemcpyDtoH_v2(host, p[4], ctypes.c_size_t(sizes[4])))
        assert min(host) == max(host) == K
        for v in p:
            ck(cu.cuMemFree_v2(v))

products()
for _ in range(2):
    ctx = ctypes.c_void_p()
    ck(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))
    products()
    ck(cu.cuCtxDestroy_v2(ctx))
products()
"""


def test_gemm_in_further_contexts_of_the_device():
    # the shared-memory limit that a kernel asks for once per device holds in every context of the process
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SECOND_CONTEXT, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ the run of them
HID, NH, DH, RD = 1024, 64, 128, 64


class Layer:
    """One layer's indexer weights, its pools, and a step through the calls in the order a server makes them."""

    def __init__(self, B, bs, stride, max_tokens, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.B, self.bs, self.stride, self.T = B, bs, stride, max_tokens
        self.gamma = 1 + 0.1 * randn(HID)
        self.w = {}
        for name, n in (("q", NH * DH), ("k", DH), ("h", NH)):
            v = randn(n, HID) / HID ** 0.5
            pad = torch.nn.functional.pad(v, (0, 0, 0, -n % 128)).view(-(-n // 128), 128, HID // 128, 128)
            sc = pad.abs().amax((1, 3)) / 448.0
            codes = (pad / sc[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, HID)[:n].contiguous()
            self.w[name] = (codes, sc.contiguous(), n)
        nblk = B * stride
        self.nblk = nblk
        self.fp4 = torch.zeros(nblk, bs, 64, dtype=torch.uint8, device="cuda")
        self.sc = torch.zeros(nblk, bs, 4, dtype=torch.uint8, device="cuda")
        self.table = torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(nblk, generator=g, device="cuda", dtype=torch.int32)
        self.rope = dev(pins._rope_table(bs * stride, RD))
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        T, i32 = max_tokens, torch.int32
        self.cached, self.new = torch.zeros(B, dtype=i32, device="cuda"), torch.zeros(B, dtype=i32, device="cuda")
        self.ctx, self.start, self.used = e(B, t=i32), e(B + 1, t=i32), e(1, t=i32)
        self.slot, self.pos = e(T, t=torch.int64), e(T, t=i32)
        self.hidden, self.resid = e(T, HID, t=torch.bfloat16), e(T, HID, t=torch.bfloat16)
        self.codes, self.scale = e(T, HID, t=torch.uint8), e(T, HID // 128)
        self.q, self.k, self.h = e(T, NH * DH, t=torch.bfloat16), e(T, DH, t=torch.bfloat16), e(T, NH)
        self.q8, self.qs = e(T, NH, DH, t=torch.uint8), e(T, NH)

    def prepare(self, n_free):
        B, T = self.B, self.T
        dsa.dsa_assign_slots(self.cached, self.new, B, self.bs, self.free, n_free, self.nblk, self.table, self.stride, T,
                             self.ctx, self.start, self.slot, self.pos, self.used)
        dsa.dsa_add_rmsnorm_e4m3(self.hidden, HID, self.resid, HID, self.gamma, 1e-6, T, HID, BF16, self.resid, None,
                                 self.codes, HID, self.scale)
        for name, out, typ in (("q", self.q, BF16), ("k", self.k, BF16), ("h", self.h, F32)):
            codes, sc, n = self.w[name]
            dsa.dsa_gemm_e4m3(self.codes, HID, self.scale, codes, HID, sc, T, n, HID, out, n, typ)
        dsa.dsa_indexer_q_rope_quant(self.q, self.pos, self.rope, self.rope.shape[0], RD, T, NH, DH, self.q8, self.qs)
        dsa.dsa_indexer_k_hadamard_mxfp4(self.k, self.slot, T, DH, self.fp4, self.sc, self.nblk * self.bs)

    def score(self, next_n, topk, max_len):
        keys = dsa.make_keys(self.fp4.view(-1, 64), None, self.table, self.bs, scale_e8m0=self.sc.view(-1, 4))
        qs = dsa.make_queries(self.B, next_n, self.ctx, max_len, True)
        ws = torch.empty(dsa.dsa_workspace_bytes(dsa.DSA_OP_LOGITS_TOPK, dsa.DSA_E4M3_MXFP4K, qs, topk), dtype=torch.uint8, device="cuda")
        idx = torch.empty(self.B * next_n, topk, dtype=torch.int32, device="cuda")
        lg = torch.empty(self.B * next_n, max_len, device="cuda")
        a = (self.q8, self.qs, dsa.DSA_E4M3_MXFP4K, self.h, NH, DH, keys, qs)
        dsa.dsa_indexer_logits(*a, lg, max_len)
        dsa.dsa_indexer_logits_topk(*a, topk, idx, None, ws, ws.numel())
        return lg, idx


def test_a_step_from_hidden_rows_to_the_selection():
    B, bs, stride, T = 3, 16, 24, 96
    ly = Layer(B, bs, stride, T, 11)
    graph = None
    lens = np.zeros(B, np.int64)
    wrote = {}                                            # pool row -> key bf16 bits
    for step, n in enumerate([32, 32, 5, 32, 1]):         # the same number of new tokens for each request
        ly.cached.copy_(torch.from_numpy(lens.astype(np.int32)))
        ly.new.fill_(n)
        ly.hidden.copy_(torch.randn(T, HID, device="cuda"))
        ly.resid.copy_(torch.randn(T, HID, device="cuda"))
        x, r = f64(ly.hidden), f64(ly.resid)
        if graph is None:                                 # the first step eagerly, the rest replayed from one capture
            ly.prepare(ly.free.shape[0])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ly.prepare(ly.free.shape[0])
        else:
            graph.replay()
        assert dsa.dsa_device_error() == 0
        lens += n
        live = B * n
        ly.free.copy_(torch.roll(ly.free, -int(ly.used)))  # the pages taken leave the list (its buffer is the graph's)
        # each link against its own reference, on what the link before gave
        slot, pos = ly.slot.cpu().numpy(), ly.pos.cpu().numpy()
        assert np.array_equal(ly.ctx.cpu().numpy(), lens) and int(ly.start[B]) == live
        assert np.array_equal(pos[:live], np.concatenate([np.arange(l - n, l) for l in lens]))
        assert len(set(slot[:live])) == live and (slot[live:] == -1).all() and not set(slot[:live]) & set(wrote)
        r64, y64 = ref.add_rmsnorm(x, r, f64(ly.gamma), float(np.float32(1e-6)), True)
        assert np.array_equal(f64(ly.resid), r64)
        ref.check_quantised(y64, ly.codes.cpu().numpy(), ly.scale.cpu().numpy(), False)
        for name, out in (("q", ly.q), ("k", ly.k), ("h", ly.h)):
            codes, sc, _ = ly.w[name]
            want, tol = ref.gemm(ly.codes.cpu().numpy(), ly.scale.cpu().numpy(), codes.cpu().numpy(), sc.cpu().numpy())
            assert (np.abs(f64(out) - want) <= tol + (0 if name == "h" else 2.0 ** -8) * (np.abs(want) + tol)).all()
        qb = ly.q.view(torch.int16).cpu().numpy().view(np.uint16).reshape(T, NH, DH)
        wc, wsc = orc.q_rope_quant(qb, pos, ly.rope.cpu().numpy(), RD)
        assert np.array_equal(ly.q8.cpu().numpy(), wc) and np.array_equal(ly.qs.cpu().numpy(), wsc)
        kb = ly.k.view(torch.int16).cpu().numpy().view(np.uint16)
        wrote.update({int(s): kb[i] for i, s in enumerate(slot[:live])})
        # the selection of this step's queries over everything cached, through the assigned pages
        lg, idx = ly.score(n, 32, int(lens.max()))
        assert dsa.dsa_device_error() == 0
        lgn = lg.cpu().numpy()
        fp4, sc8, table = ly.fp4.cpu().numpy(), ly.sc.cpu().numpy(), ly.table.cpu().numpy()
        want = orc.indexer_logits(ly.q8[:live].cpu().numpy(), ly.qs[:live].cpu().numpy(), "e4m3", ly.h[:live].cpu().numpy(),
                                  fp4.reshape(-1, 64), sc8.reshape(-1, 4), table, bs, B, n, lens.astype(np.int32), True,
                                  k_dtype="mxfp4")
        parity.assert_logits_close(lgn, want)
        parity.assert_topk_exact(idx.cpu().numpy(), lgn, 32)
    # every key written since the start still stands in its row
    rows = np.array(sorted(wrote))
    w_fp4, w_sc = orc.k_hadamard_mxfp4(np.stack([wrote[s] for s in rows]), rows, np.zeros_like(fp4), np.zeros_like(sc8))
    assert np.array_equal(sc8, w_sc)
    assert (fp4 != w_fp4).mean() <= 0.01                  # codes at a rounding boundary
