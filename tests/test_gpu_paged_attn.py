"""dsa_paged_attn against the definition in 64 bits (dense_ref.attention, where the bounds are derived).  Everything that
no row may see is poisoned: NaN behind a sequence's last key and in unused pages, block ids out of range in the table
entries that are not to be read."""
import math

import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from deepseek_v4_sparse_dsa_gb300 import dsa  # noqa: E402


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Case:
    def __init__(self, new, lens, H, Hkv, D, bs=16, causal=True, window=0, sink=False, seed=0, head_major=False, shared=False,
                 pad=0, gap=0, spare=1, scale=None):
        g = gen(seed)
        self.__dict__.update(new=new, lens=lens, H=H, Hkv=Hkv, D=D, bs=bs, causal=causal, window=window)
        B, self.B = len(new), len(new)
        self.start = torch.tensor([gap + sum(new[:b]) for b in range(B + 1)], device="cuda", dtype=torch.int32)
        self.gap, self.used = gap, sum(new)
        self.T = gap + self.used + spare                   # rows before the first sequence and behind the last
        self.ctx = torch.tensor(lens, device="cuda", dtype=torch.int32)
        pages = [-(-n // bs) for n in lens]
        self.stride = max(pages + [1]) + 1
        self.num_blocks = sum(pages) + 3
        pool = torch.randperm(self.num_blocks, generator=g, device="cuda", dtype=torch.int32)
        self.table = torch.full((B, self.stride), 1 << 30, device="cuda", dtype=torch.int32)
        shape = (self.num_blocks, Hkv, bs, D) if head_major else (self.num_blocks, bs, Hkv, D)
        kc, vc = (torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        if head_major:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        if shared:
            vc = kc
        self.k_rows, self.v_rows, self.kc, self.vc = [], [], kc, vc
        at = 0
        for b in range(B):
            L, n = lens[b], new[b]
            k = torch.randn(L, Hkv, D, device="cuda", generator=g).bfloat16()
            v = k if shared else torch.randn(L, Hkv, D, device="cuda", generator=g).bfloat16()
            first = max(0, L - n - window + 1) if window and n else 0    # the oldest key that a row sees
            if n == 0:
                first = L
            for pg in range(pages[b]):
                blk = int(pool[at + pg])
                lo, hi = pg * bs, min(L, (pg + 1) * bs)
                if hi <= first:
                    continue                               # nobody sees the page: it and its entry stay poisoned
                self.table[b, pg] = blk
                lo2 = max(lo, first)
                kc[blk, lo2 - lo:hi - lo] = k[lo2:hi]
                vc[blk, lo2 - lo:hi - lo] = v[lo2:hi]
            at += pages[b]
            self.k_rows.append(k)
            self.v_rows.append(v)
        self.ldq = H * D + pad
        self.q = torch.full((self.T, self.ldq), float("nan"), device="cuda", dtype=torch.bfloat16)
        self.rows = slice(gap, gap + self.used)
        self.q[self.rows, :H * D] = torch.randn(self.used, H * D, device="cuda", generator=g).mul_(2).bfloat16()
        self.sink = torch.randn(H, device="cuda", generator=g) if sink else None
        self.scale = D ** -0.5 if scale is None else scale
        self.out = torch.full((self.T, self.ldq), -7.0, device="cuda", dtype=torch.bfloat16)
        self.lse = torch.full((self.T, H), -7.0, device="cuda")
        self.ws = torch.full((dsa.dsa_paged_attn_workspace_bytes(self.T, B, H, Hkv, D),), 255, device="cuda", dtype=torch.uint8)

    def run(self, stream=None, lse=True):
        dsa.dsa_paged_attn(self.q, self.ldq, self.T, self.H, self.Hkv, self.D, self.start, self.ctx, self.B, self.table,
                           self.stride, dsa.make_kv_cache(self.kc, self.vc), self.scale, self.causal, self.window, self.sink,
                           self.out, self.ldq, self.lse if lse else None, self.ws, self.ws.numel(), stream)

    def want(self):
        q = self.q[self.rows, :self.H * self.D].reshape(self.used, self.H, self.D)
        return ref.attention(q, self.k_rows, self.v_rows, self.new, self.lens, self.scale, self.causal, self.window, self.sink)

    def compare(self, wanted):
        out, lse, out_tol, lse_tol = wanted
        HD = self.H * self.D
        got = self.out[self.rows, :HD].double().reshape(out.shape)
        err = (got - out).abs()
        assert bool((err <= out_tol).all()), (float((err / out_tol.clamp(min=1e-30)).nan_to_num(1e9).max()), int((~(err <= out_tol)).sum()))
        l = self.lse[self.rows].double()
        assert torch.equal(l == -math.inf, lse == -math.inf)
        fin = lse > -math.inf
        le = (l - lse).abs()[fin]
        assert bool((le <= lse_tol[fin]).all()), float((le / lse_tol[fin]).max())
        # rows of no sequence, and what lies between the rows
        assert bool((self.out[:self.gap] == -7).all()) and bool((self.out[self.gap + self.used:] == -7).all())
        assert bool((self.out[:, HD:] == -7).all())
        assert bool((self.lse[:self.gap] == -7).all()) and bool((self.lse[self.gap + self.used:] == -7).all())

    def check(self):
        self.run()
        assert dsa.dsa_device_error() == 0
        self.compare(self.want())
        return self


SMALL = [  # new tokens and lengths of each sequence
    ([1], [1]), ([1], [128]), ([1], [129]), ([3], [3]), ([1, 1, 1], [5, 700, 64]), ([16], [16]), ([17], [145]), ([2, 0, 5], [300, 50, 5]),
    ([40, 1], [40, 1000]), ([33, 64, 1], [900, 64, 257]),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(8, 1), (8, 8), (6, 2), (64, 1)])
@pytest.mark.parametrize("lengths", SMALL)
def test_small(lengths, heads, D):
    new, lens = lengths
    for i, kw in enumerate([dict(), dict(causal=False, sink=True, bs=20), dict(window=37, bs=1, sink=True), dict(window=128, bs=256, head_major=True)]):
        Case(new, lens, *heads, D, seed=i, **kw).check()


@pytest.mark.parametrize("D", [64, 128])
def test_long_rows_are_cut(D):
    # one token over a long context: every SM has a piece of it
    Case([1], [20000], 16, 2, D, bs=64).check()
    Case([2, 1], [70000, 300], 64, 1, D, bs=64, sink=True, seed=1).check()
    Case([1, 1, 1, 1], [9000, 1, 4097, 128], 8, 8, D, bs=128, seed=2).check()
    Case([1] * 3, [30000] * 3, 12, 4, D, bs=64, window=5000, sink=True, seed=3).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(8, 1), (12, 4), (5, 5), (64, 1)])
def test_chunks_of_prompts(heads, D):
    Case([700], [700], *heads, D).check()
    Case([300, 1, 513, 0, 90], [1300, 900, 513, 77, 4000], *heads, D, bs=64, seed=1, sink=True).check()
    Case([600, 200], [1500, 200], *heads, D, bs=64, window=300, seed=2).check()
    Case([257], [3000], *heads, D, bs=8, causal=False, seed=3).check()


def test_more_key_heads_than_pieces_and_wide_groups():
    Case([3, 2], [50, 400], 128, 64, 64, seed=1).check()
    Case([2, 1], [50, 400], 600, 2, 64, seed=2).check()      # 300 rows per token: more than a row block
    Case([2, 1], [50, 400], 130, 1, 128, seed=3).check()


def test_no_new_tokens_and_many_key_heads():
    c = Case([0, 0], [5, 9], 8, 2, 64).check()               # nothing to do: nothing is written
    assert bool((c.out == -7).all())
    Case([2, 1], [30, 200], 260, 260, 64, bs=8, seed=1).check()
    Case([1], [3000], 520, 130, 128, bs=64, sink=True, seed=2).check()


def test_plan_of_many_sequences():
    # more sequences, and more row blocks, than a CTA plans by itself
    new = [i % 3 for i in range(1500)]
    Case(new, [n + (7 * i) % 200 for i, n in enumerate(new)], 4, 1, 64, seed=1).check()
    c = Case([1200], [1300], 300, 1, 64, seed=2)
    assert c.T * 300 // 256 > 1024
    c.check()
    c = Case([1] * 1100, [(5 * i) % 90 + 1 for i in range(1100)], 2, 2, 128, window=30, sink=True, seed=3)
    c.check()


def test_rows_that_see_nothing():
    # more new tokens than keys: the first ones sit before position 0; a sequence without keys; a window that is empty
    c = Case([10, 4, 2], [4, 0, 6], 8, 2, 64)
    c.check()
    assert bool((c.out[:6, :512] == 0).all()) and bool((c.lse[:6] == -math.inf).all())
    c = Case([10, 4, 2], [4, 0, 6], 8, 2, 128, sink=True)
    c.check()
    assert torch.equal(c.lse[10:14], c.sink.expand(4, 8)) and bool((c.out[10:14, :1024] == 0).all())


@pytest.mark.parametrize("new, lens", [([1, 4], [20000, 2]), ([200, 3], [9000, 1])])      # cut and whole items, empty rows
def test_sinks_without_a_finite_form_in_base_2(new, lens):
    c = Case(new, lens, 4, 2, 128, bs=64)
    c.check()                                                # no sinks
    out, lse = (x[c.rows].clone() for x in (c.out, c.lse))
    low = torch.finfo(torch.float32).min
    c.sink = torch.tensor([math.inf, -math.inf, low, math.nan], device="cuda")
    for gone in (False, True):
        if gone:                                             # every page's entry is bad: all rows see nothing
            c.table.fill_(-1)
            out.zero_()
            lse.fill_(-math.inf)
        c.run()
        assert dsa.dsa_device_error() == (dsa.DSA_DEVERR_INDEX if gone else 0)
        got, l = c.out[c.rows].view(-1, 4, 128), c.lse[c.rows]
        assert bool((got[:, 0] == 0).all()) and bool((l[:, 0] == math.inf).all())
        assert bool(got[:, 3].isnan().all()) and bool(l[:, 3].isnan().all())
        assert torch.equal(got[:, 1:3], out.view(-1, 4, 128)[:, 1:3])          # e^sink is nothing next to any score
        assert torch.equal(l[:, 1], lse[:, 1])
        assert torch.equal(l[:, 2], lse[:, 2].clamp(min=low))


def test_strides_gaps_and_shared_keys_and_values():
    Case([5, 70], [200, 70], 8, 2, 128, pad=24, gap=3, spare=9, head_major=True, sink=True).check()
    Case([5, 70], [200, 300], 16, 1, 128, shared=True, bs=64, pad=8, gap=1).check()
    c = Case([2], [40], 4, 2, 64, seed=3)
    wide = torch.full((c.num_blocks, c.bs, 5, 64), float("nan"), device="cuda", dtype=torch.bfloat16)   # heads 1 and 3 of 5
    for i in range(2):
        wide[:, :, 2 * i + 1] = c.kc[:, :, i]
    c.kc, old = wide[:, :, 1::2], c.vc
    wide_v = torch.full_like(wide, float("nan"))
    for i in range(2):
        wide_v[:, :, 2 * i + 1] = old[:, :, i]
    c.vc = wide_v[:, :, 1::2]
    c.check()


def test_no_lse_and_large_scale():
    c = Case([3, 200], [1000, 200], 8, 2, 128, scale=1.0)    # scores of tens: the running maximum moves often
    c.check()
    out = c.out.clone()
    c.out.fill_(-7)
    c.lse.fill_(-7)
    c.run(lse=False)
    assert torch.equal(c.out, out) and bool((c.lse == -7).all())


def test_rising_scores_move_the_maximum():
    # every key tile's maximum exceeds the last one's by far
    c = Case([1, 150], [1000, 1000], 8, 1, 64, bs=64, scale=1.0)
    for b in range(2):
        up = torch.linspace(0, 60, 1000, device="cuda")[:, None, None]
        k = (c.k_rows[b].float() * 0.1 + up / 64).bfloat16()
        c.k_rows[b].copy_(k)
        for pg in range(-(-1000 // 64)):
            n = min(64, 1000 - 64 * pg)
            c.kc[int(c.table[b, pg]), :n] = k[64 * pg:64 * pg + n]
    c.q.abs_()
    c.check()


def put(c, b, pos, k=None, v=None, dim=3):
    blk = int(c.table[b, pos // c.bs])
    for val, cache, rows in ((k, c.kc, c.k_rows), (v, c.vc, c.v_rows)):
        if val is not None:
            cache[blk, pos % c.bs, :, dim] = val
            rows[b][pos, :, dim] = val


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [6, 170])
def test_what_a_row_does_not_see_never_touches_it(new, D):
    # a key and a value that are no numbers, at the last-but-two position: rows before it are what they are without
    for bad in (float("nan"), float("inf"), -float("inf")):
        clean, c = (Case([new, 2], [400, 300], 8, 2, D, seed=5) for _ in range(2))
        clean.check()
        put(c, 0, 397, v=bad)
        c.run()
        row = 397 - (400 - new)                              # the first row that sees it
        a, b = (x.out[:, :8 * D].view(-1, 8, D) for x in (clean, c))
        assert torch.equal(a[:row], b[:row]) and torch.equal(a[new:new + 2], b[new:new + 2])
        seen = b[row:new]
        assert bool((seen[..., 3].isnan() if bad != bad else seen[..., 3] == bad).all())
        rest = [d for d in range(D) if d != 3]
        assert torch.equal(seen[..., rest], a[row:new][..., rest])
        assert torch.equal(clean.lse, c.lse)
        c = Case([new, 2], [400, 300], 8, 2, D, seed=5)
        put(c, 0, 397, k=bad)
        c.run()
        b = c.out[:, :8 * D].view(-1, 8, D)
        assert torch.equal(a[:row], b[:row]) and torch.equal(a[new:new + 2], b[new:new + 2])
        assert torch.equal(clean.lse[:row], c.lse[:row])
        if bad != bad:
            assert bool(b[row:new].isnan().all()) and bool(c.lse[row:new].isnan().all())
    assert dsa.dsa_device_error() == 0


def test_what_left_the_window_never_touches_a_row():
    new, L, w = 40, 600, 100
    clean, c = (Case([new], [L], 8, 2, 64, window=w, seed=6) for _ in range(2))
    clean.run()
    put(c, 0, 480, v=float("nan"))                           # seen by the tokens up to position 579
    c.run()
    last = 480 + w - 1 - (L - new)
    a, b = (x.out[:, :512].view(-1, 8, 64) for x in (clean, c))
    assert torch.equal(a[last + 1:new], b[last + 1:new]) and bool(b[:last + 1, :, 3].isnan().all())
    assert dsa.dsa_device_error() == 0


def test_a_value_that_is_no_number_in_a_cut_row():
    c = Case([2], [30000], 8, 1, 128, bs=64, seed=7)
    clean = Case([2], [30000], 8, 1, 128, bs=64, seed=7)
    clean.run()
    put(c, 0, 29999, v=float("inf"))                         # the second token's own
    put(c, 0, 123, v=-float("inf"), dim=5)                   # seen by both
    c.run()
    a, b = (x.out[:2, :1024].view(2, 8, 128) for x in (clean, c))
    assert bool((b[1, :, 3] == float("inf")).all()) and bool((b[:, :, 5] == -float("inf")).all())
    assert torch.equal(a[0, :, 3], b[0, :, 3])
    rest = [d for d in range(128) if d not in (3, 5)]
    assert torch.equal(a[..., rest], b[..., rest])


def test_queries_that_are_no_numbers_stay_in_their_row():
    clean, c = (Case([9], [300], 8, 2, 64, seed=8) for _ in range(2))
    clean.run()
    c.q[4, 70] = float("nan")                                # head 1
    c.run()
    a, b = (x.out[:9, :512].view(9, 8, 64) for x in (clean, c))
    assert bool(b[4, 1].isnan().all()) and bool(c.lse[4, 1].isnan())
    keep = torch.ones(9, 8, dtype=torch.bool, device="cuda")
    keep[4, 1] = False
    assert torch.equal(a[keep], b[keep])


def test_bad_blocks_mask_their_keys():
    for D, new in ((64, 3), (128, 140)):
        c = Case([new, 1], [500, 40], 8, 2, D, bs=16, seed=9)
        for pg, bad in ((3, -1), (20, c.num_blocks), (30, 1 << 30)):
            c.table[0, pg] = bad
            c.k_rows[0][16 * pg:16 * (pg + 1)] = float("nan")     # dense_ref: a masked key
        c.run()
        assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
        c.compare(c.want())


def test_keys_past_the_table_and_bad_lengths():
    c = Case([2, 3], [100, 90], 4, 2, 64, bs=16)
    c.stride = 5                                             # 80 keys
    c.table = c.table[:, :5].contiguous()
    for b in range(2):
        c.k_rows[b][80:] = float("nan")
    c.run()
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    c.compare(c.want())
    c = Case([2, 3, 1], [100, 90, 8], 4, 2, 64)
    good = c.start.clone()
    c.ctx[0] = -5
    c.run()
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    assert bool((c.out[:2, :256] == 0).all())
    for starts in ([0, 2, 5, 600], [0, -3, 5, 6], [4, 2, 5, 6]):   # past T, negative, descending: left out
        c.out.fill_(-7)
        c.start.copy_(torch.tensor(starts, device="cuda", dtype=torch.int32))
        c.ctx.copy_(torch.tensor([100, 90, 8], device="cuda", dtype=torch.int32))
        c.run()
        assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
    c.start.copy_(good)
    c.lse.fill_(-7)
    c.out.fill_(-7)
    c.check()
    # ranges that overlap so often that they would need more row blocks than there can be
    c = Case([4] * 40, [10] * 40, 4, 2, 64, seed=2)
    c.start.copy_(torch.tensor([0, c.T] * 20 + [0], device="cuda", dtype=torch.int32))
    c.run()
    assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX


def test_far_cache_rows():
    # a pool of more than 2^31 elements, the sequence's pages at its end
    D, bs, Hkv = 128, 64, 2
    blocks = (1 << 31) // (bs * Hkv * D) + 8
    c = Case([2], [300], 8, Hkv, D, bs=bs, seed=10)
    kc, vc = (torch.zeros(blocks, bs, Hkv, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc[-c.num_blocks:], vc[-c.num_blocks:] = c.kc, c.vc
    live = c.table < c.num_blocks
    c.table[live] += blocks - c.num_blocks
    c.kc, c.vc = kc, vc
    c.check()


def test_same_batch_same_bits_and_any_workspace():
    c = Case([1, 200, 3], [9000, 900, 400], 8, 2, 128, bs=64, seed=11).check()
    out, lse = c.out.clone(), c.lse.clone()
    for fill in (0, 255, 127):
        c.ws.fill_(fill)
        c.out.fill_(-7)
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_two_streams_at_once_and_a_captured_graph():
    cases = [Case([1, 1, 2], [9000, 100, 3000], 8, 2, 128, seed=12), Case([300], [800], 8, 1, 64, seed=13)]
    for c in cases:
        c.check()
    want = [(c.out.clone(), c.lse.clone()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                c.out.fill_(-7)
                c.run(st)
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cases, want):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    # captured: the lengths are read when the graph runs, not when it is made
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for lens in ([9000, 100, 3000], [5000, 33, 2], [1, 1, 2]):
        c.ctx.copy_(torch.tensor(lens, device="cuda", dtype=torch.int32))
        c.out.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.lens, d.k_rows, d.v_rows = lens, [k[:n] for k, n in zip(c.k_rows, lens)], [v[:n] for v, n in zip(c.v_rows, lens)]
        d.compare(d.want())
    assert dsa.dsa_device_error() == 0


def test_a_layer_step():
    # slots -> table -> norm + rotation + cache write -> attention -> rotation of the output taken back, for a batch whose
    # sequences grow over two steps; against the whole computed in 64 bits from the projections
    H, Hkv, D, bs, R = 8, 2, 128, 16, 64
    g = gen(20)
    blocks = 40
    free = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    B, stride = 3, 12
    i32 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.int32)  # noqa: E731
    table, cs = i32(B, stride) - 1, torch.empty(256, R, device="cuda")
    kc, vc = (torch.full((blocks, bs, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gq, gk = (1 + 0.1 * torch.randn(D, device="cuda", generator=g) for _ in range(2))
    dsa.dsa_rope_table(dsa.make_rope_params(scaling=dsa.DSA_ROPE_YARN, factor=4.0, original_max_pos=64.0), R, 0, 256, cs)
    cached, used = [0, 0, 0], 0
    history = [torch.empty(0, (H + 2 * Hkv) * D, device="cuda") for _ in range(B)]
    for new in ([37, 5, 0], [1, 20, 1], [1, 1, 1]):
        T = sum(new) + 2                                     # two rows of padding
        ctx, start, slot, pos, n_used = i32(B), i32(B + 1), torch.empty(T, device="cuda", dtype=torch.int64), i32(T), i32(1)
        c, n = (torch.tensor(v, device="cuda", dtype=torch.int32) for v in (cached, new))
        dsa.dsa_assign_slots(c, n, B, bs, free[used:], blocks - used, blocks, table, stride, T, ctx, start, slot, pos, n_used)
        used += int(n_used)
        qkv = torch.randn(T, (H + 2 * Hkv) * D, device="cuda", generator=g).bfloat16()
        ld, q = qkv.stride(0), torch.empty(T, H * D, device="cuda", dtype=torch.bfloat16)
        dsa.dsa_qk_norm_rope(qkv, ld, H, qkv[:, H * D:], ld, Hkv, qkv[:, (H + Hkv) * D:], ld, T, D, dsa.DSA_REAL_BF16, gq, gk,
                             1e-6, pos, cs, 256, R, D - R, dsa.DSA_ROPE_INTERLEAVED, q, H * D, None, 0,
                             dsa.make_kv_cache(kc, vc), slot)
        out = torch.zeros_like(q)
        ws = torch.empty(dsa.dsa_paged_attn_workspace_bytes(T, B, H, Hkv, D), device="cuda", dtype=torch.uint8)
        dsa.dsa_paged_attn(q, H * D, T, H, Hkv, D, start, ctx, B, table, stride, dsa.make_kv_cache(kc, vc), D ** -0.5, True, 0,
                           None, out, H * D, None, ws, ws.numel())
        back = torch.empty_like(out)
        dsa.dsa_rope(out, H * D, D, pos, cs, 256, R, D - R, dsa.DSA_ROPE_INTERLEAVED, True, T, H, D, dsa.DSA_REAL_BF16, back,
                     H * D, D)
        assert dsa.dsa_device_error() == 0
        at = 0
        for b in range(B):
            history[b] = torch.cat([history[b], qkv[at:at + new[b]].float()])
            x = history[b].double().view(-1, H + 2 * Hkv, D)
            p = torch.arange(len(x), device="cuda")
            qr = ref.rotate(ref.norm(x[:, :H], gq, 1e-6), cs[p], R, D - R, False)[0]
            kr = ref.rotate(ref.norm(x[:, H:H + Hkv], gk, 1e-6), cs[p], R, D - R, False)[0].repeat_interleave(H // Hkv, 1)
            v = x[:, H + Hkv:].repeat_interleave(H // Hkv, 1)
            s = torch.einsum("nhd,lhd->hnl", qr, kr) * D ** -0.5
            s = s.masked_fill(p[None, None, :] > p[None, :, None], -math.inf)
            o = torch.einsum("hnl,lhd->nhd", s.softmax(-1), v)
            o = ref.rotate(o, cs[p], R, D - R, False, True)[0][len(x) - new[b]:]
            got = back[at:at + new[b]].double().view(-1, H, D)
            # q, k, the output and its rotation are each rounded to bf16: scores off by 2 x 2^-8 of |q||k| D^-1/2 at most
            # (about 0.1 here), seen through the mean of |v| below 4.5
            if new[b]:
                assert float((got - o).norm() / o.norm()) <= 2.0 ** -5
                assert float((got - o).abs().max()) <= 0.5
            at += new[b]
        cached = [a + b for a, b in zip(cached, new)]


def test_many_calls_in_a_row():
    # calls one behind the other, whose CTAs start as soon as the last ones' leave, with pieces of few tiles, all rows of
    # a tile in use, and windows: nothing waits for what has already passed, and nothing changes
    cases = [Case([2] * 32, [4096 * (b + 1) for b in range(32)], 64, 1, 128, bs=64, window=4096, sink=True, seed=1),
             Case([1] * 40, [100 + 37 * b for b in range(40)], 64, 1, 64, bs=16, seed=2),
             Case([130, 7, 64], [300, 70, 640], 6, 2, 128, bs=20, seed=3)]
    for c in cases:
        c.check()
        out, lse = c.out.clone(), c.lse.clone()
        for _ in range(100):
            c.run()
        assert dsa.dsa_device_error() == 0
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_gathered_pages_of_any_size():
    # page sizes that no copy of several rows fits: 1, 3, 12 and 100 rows; heads side by side, apart, and within a row
    for i, bs in enumerate((1, 3, 12, 100)):
        for D in (64, 128):
            Case([3, 150], [500, 400], 8, 2, D, bs=bs, seed=i, head_major=bool(i % 2), window=0 if i < 2 else 170).check()


@pytest.mark.parametrize("case", [dict(new=[1, 1, 3], lens=[9000, 100, 3000], H=8, Hkv=2, D=128, bs=64),
                                  dict(new=[1] * 12, lens=[50000] * 12, H=16, Hkv=4, D=128, bs=64),
                                  dict(new=[300, 40], lens=[800, 700], H=8, Hkv=1, D=64, bs=16),
                                  dict(new=[300, 40], lens=[800, 700], H=6, Hkv=2, D=128, bs=20, window=100)])
def test_expired_waits_are_told_and_leave_the_context_usable(case):
    c = Case(**case).check()
    right, told = c.out.clone(), 0
    for limit in (1, 1000, 5000, 1):
        dsa.dsa_set_wait_limit_ns(limit)
        try:
            for _ in range(2):
                c.run()                                      # the sums of parts then read whatever is there
            err = dsa.dsa_device_error()
        finally:
            dsa.dsa_set_wait_limit_ns(0)
        # (the clock ticks less often than some waits last: a call all of whose waits were short is a right one)
        assert err in (0, dsa.DSA_DEVERR_TIMEOUT) and (err or torch.equal(c.out, right))
        told |= err
    assert told or sum(case["lens"]) < 100000                # work of many microseconds does not pass unnoticed
    c.out.fill_(-7)
    c.lse.fill_(-7)
    c.ws.fill_(255)
    c.check()


# ------------------------------------------------------------------ workspaces, ranges that are none, the error as a whole
@pytest.mark.parametrize("D, heads", [(128, (64, 8)), (64, (8, 1)), (64, (6, 2))])
def test_a_workspace_of_a_larger_step_fits_every_smaller_one(D, heads):
    # a decode batch's buffer serves a chunk of one sequence (whose own size, with two row tiles, is larger) and the
    # other way round, with either form's results
    H, Hkv = heads
    big = dsa.dsa_paged_attn_workspace_bytes(300, 300, H, Hkv, D)
    assert dsa.dsa_paged_attn_workspace_bytes(250, 1, H, Hkv, D) > big
    for i, (new, lens) in enumerate([([249], [2000]), ([16] * 10, [700] * 10), ([1], [5000]), ([100, 3, 0], [100, 9000, 7]),
                                     ([280], [280])]):
        c = Case(new, lens, H, Hkv, D, bs=64, seed=i, sink=bool(i % 2))
        assert c.T <= 300 and c.B <= 300
        c.check()
        c.ws = torch.full((big,), 255, device="cuda", dtype=torch.uint8)
        c.out.fill_(-7)
        c.lse.fill_(-7)
        c.check()
        again = c.out.clone()
        c.run()
        assert torch.equal(c.out, again)
    with pytest.raises(dsa.DsaError) as e:
        c.ws = c.ws[:1 << 20]
        c.run()
    assert e.value.status == dsa.DSA_ERR_WORKSPACE
    # a chunk's buffer serves a decode batch
    big = dsa.dsa_paged_attn_workspace_bytes(4096, 64, H, Hkv, D)
    c = Case([1] * 60, [90 * b + 1 for b in range(60)], H, Hkv, D, bs=64, seed=9)
    assert c.ws.numel() <= big


def test_a_workspace_of_many_sequences_serves_one_long_chunk():
    # row blocks of 128 rows, more than a CTA plans by itself
    c = Case([1100], [1300], 64, 1, 64, seed=1).check()
    size = dsa.dsa_paged_attn_workspace_bytes(c.T, c.T, 64, 1, 64)
    assert size < c.ws.numel() and c.T * 64 // 128 > 512
    c.ws = torch.full((size,), 255, device="cuda", dtype=torch.uint8)
    c.out.fill_(-7)
    c.lse.fill_(-7)
    c.check()


def test_ranges_that_are_none_are_left_out():
    # each sequence whose rows are no range of the T rows is left out, the others get what they always get, and a row of
    # no sequence stays as it was
    q_rows, lens = 8, [100, 90, 60]
    for starts in ([0, 2, 5, 600], [0, -3, 5, 6], [4, 2, 5, 6], [0, 3, 1, 7], [7, 7, 7, 9], [-1, 2, 2, 8], [0, 8, 0, 8]):
        c = Case([3, 3, 2], lens, 4, 2, 64, seed=4, spare=0)
        assert c.T == q_rows
        c.start = torch.tensor(starts, device="cuda", dtype=torch.int32)
        c.run()
        assert dsa.dsa_device_error() == dsa.DSA_DEVERR_INDEX
        owner = [[b for b in range(3) if starts[b] <= t < starts[b + 1] and 0 <= starts[b] and starts[b + 1] <= q_rows]
                 for t in range(q_rows)]
        out, lse = c.out.view(q_rows, 4, 64), c.lse
        for t in range(q_rows):
            if not owner[t]:
                assert bool((out[t] == -7).all()) and bool((lse[t] == -7).all())
        for b in range(3):
            s, e = starts[b], starts[b + 1]
            rows = [t for t in range(max(s, 0), max(e, 0)) if t < q_rows and owner[t] == [b]]
            if not rows:
                continue
            q = c.q[s:e].reshape(e - s, 4, 64)
            want = ref.attention(q, [c.k_rows[b]], [c.v_rows[b]], [e - s], [lens[b]], c.scale, True, 0, None)
            at = [t - s for t in rows]
            assert bool(((out[rows].double() - want[0][at]).abs() <= want[2][at]).all())
            assert bool(((lse[rows].double() - want[1][at]).abs() <= want[3][at]).all())


@pytest.mark.parametrize("new, lens, kw", [
    ([1] * 8, [4096 * (b + 1) for b in range(8)], dict(H=16, Hkv=2, D=128, bs=64)),
    ([256], [20000], dict(H=16, Hkv=2, D=128, bs=64)),
    ([1500, 30], [1500, 9000], dict(H=8, Hkv=2, D=64, bs=16)),
    ([2] * 6, [9000] * 6, dict(H=64, Hkv=1, D=128, bs=64, window=4096, sink=True)),
])
def test_the_norm_of_the_error(new, lens, kw):
    # Per element the bound of dense_ref is worst case; as a whole the roundings are as often up as down.  A rounding to
    # bf16 is off by at most 2^-8 of the value, evenly spread: 2^-8 / sqrt(3) in the mean square.  The output has its own;
    # the weights' adds sum_j p_j d_j v_j, whose mean square, for values v_j of either sign, is d^2 of the output's own
    # sum_j p_j v_j.  Together at most sqrt(2) 2^-8 / sqrt(3) = 3.19e-3 of the norm.  A value that is lost or taken twice
    # among n even weights is 1 / sqrt(n) of it.
    c = Case(new, lens, seed=5, **kw)
    c.run()
    assert dsa.dsa_device_error() == 0
    out = c.want()[0]
    err = c.out[c.rows, :c.H * c.D].double().reshape(out.shape) - out
    assert float(err.norm() / out.norm()) <= math.sqrt(2.0 / 3) * 2.0 ** -8
