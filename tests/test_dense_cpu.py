"""The dense-attention calls on a machine without a GPU: bad arguments are refused on the host before any launch, empty
calls are accepted, and the cache structure is filled from tensors' strides."""
import pytest

from deepseek_v4_sparse_dsa_gb300 import dsa

BF16, F32 = dsa.DSA_REAL_BF16, dsa.DSA_REAL_F32
INVALID, UNSUPPORTED, WORKSPACE = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE
P = [0x10000000 * (i + 1) for i in range(16)]                # addresses that are never touched


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from deepseek_v4_sparse_dsa_gb300 import build
    if not os.path.exists(dsa.LIB_PATH):
        build.build()
    return dsa.load()


def refused(call, status, **kw):
    before = dsa.dsa_launch_count()
    with pytest.raises(dsa.DsaError) as e:
        call(**kw)
    assert e.value.status == status
    assert dsa.dsa_launch_count() == before


def table(params=None, R=64, pos0=0, n=16, out=P[0], **p):
    dsa.dsa_rope_table(params or dsa.make_rope_params(**p), R, pos0, n, out, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), INVALID), (dict(R=63), INVALID), (dict(R=-2), INVALID), (dict(R=258), UNSUPPORTED), (dict(n=-1), INVALID),
    (dict(pos0=-1), INVALID), (dict(pos0=1 << 31, n=1), UNSUPPORTED), (dict(n=(1 << 31) + 1), UNSUPPORTED),
    (dict(pos0=1 << 62, n=1 << 62), UNSUPPORTED), (dict(out=None), INVALID), (dict(out=P[0] + 2), INVALID),
    (dict(base=1.0), INVALID), (dict(base=-3.0), INVALID), (dict(base=float("nan")), INVALID),
    (dict(base=float("inf")), INVALID), (dict(amplitude=float("nan")), INVALID), (dict(scaling=3), INVALID),
    (dict(scaling=1, factor=0.5), INVALID), (dict(scaling=2, factor=float("inf")), INVALID),
    (dict(scaling=2, factor=2.0, original_max_pos=0.0), INVALID), (dict(scaling=2, factor=2.0, beta_slow=0.0), INVALID),
    (dict(scaling=2, factor=2.0, beta_fast=1.0, beta_slow=2.0), INVALID),
    (dict(scaling=2, factor=2.0, beta_fast=float("inf")), INVALID),
])
def test_table_refusals(kw, status):
    refused(table, status, **kw)


def rope(x=P[0], ldx=512, hx=128, pos=P[1], cs=P[2], max_pos=100, R=64, off=0, layout=0, inverse=False, T=4, H=4, D=128, type=BF16,
         y=P[3], ldy=512, hy=128):
    dsa.dsa_rope(x, ldx, hx, pos, cs, max_pos, R, off, layout, inverse, T, H, D, type, y, ldy, hy, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(D=0), INVALID), (dict(R=0), INVALID),
    (dict(R=63), INVALID), (dict(R=130), INVALID), (dict(off=-2), INVALID), (dict(off=65), INVALID), (dict(off=2**31 - 1), INVALID),
    (dict(D=257), UNSUPPORTED), (dict(T=1 << 30, H=4), UNSUPPORTED), (dict(T=1 << 40), UNSUPPORTED), (dict(layout=2), INVALID),
    (dict(max_pos=-1), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID),
    (dict(cs=None), INVALID), (dict(x=P[0] + 1), INVALID), (dict(type=F32, y=P[3] + 2), INVALID), (dict(pos=P[1] + 2), INVALID),
    (dict(cs=P[2] + 2), INVALID), (dict(hx=127), INVALID), (dict(hy=100), INVALID), (dict(ldx=100), INVALID), (dict(ldy=127), INVALID),
    (dict(y=P[0], ldy=520), INVALID), (dict(y=P[0], hy=136), INVALID), (dict(y=P[1]), INVALID), (dict(y=P[2]), INVALID),
])
def test_rope_refusals(kw, status):
    refused(rope, status, **kw)


def qk(q=P[0], ldq=768, H=4, k=P[1], ldk=768, Hkv=1, v=P[2], ldv=768, T=4, D=128, type=BF16, gq=P[3], gk=P[4], eps=1e-6, pos=P[5],
       cs=P[6], max_pos=100, R=64, off=0, layout=0, qo=P[7], ldqo=512, ko=None, ldko=0, kc=P[8], vc=P[9], slot=P[10], **kv):
    args = dict(num_blocks=8, block_size=16, block_stride=2048, row_stride=128, head_stride=128)
    args.update(kv)
    dsa.dsa_qk_norm_rope(q, ldq, H, k, ldk, Hkv, v, ldv, T, D, type, gq, gk, eps, pos, cs, max_pos, R, off, layout, qo, ldqo, ko,
                         ldko, dsa.dsa_kv_cache(kc, vc, *args.values()), slot, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(type=7), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(D=0), INVALID),
    (dict(D=258), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(T=1 << 50), UNSUPPORTED), (dict(R=-2), INVALID),
    (dict(R=3), INVALID), (dict(R=130), INVALID), (dict(off=66), INVALID), (dict(layout=-1), INVALID), (dict(pos=None), INVALID),
    (dict(cs=None), INVALID), (dict(gk=None), INVALID), (dict(gq=None), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(ldq=511), INVALID),
    (dict(ldqo=511), INVALID), (dict(k=None), INVALID), (dict(ldk=127), INVALID), (dict(ldv=127), INVALID),
    (dict(kc=None), INVALID), (dict(ko=P[11], ldko=127), INVALID), (dict(vc=None), INVALID), (dict(slot=None), INVALID),
    (dict(slot=P[10] + 4), INVALID), (dict(kc=P[8] + 1), INVALID), (dict(num_blocks=-1), INVALID), (dict(block_size=0), INVALID),
    (dict(row_stride=127), INVALID), (dict(block_stride=0), INVALID), (dict(H=4, Hkv=2, ldk=768, head_stride=64), INVALID),
    (dict(num_blocks=1 << 31), UNSUPPORTED), (dict(block_stride=1 << 39), UNSUPPORTED), (dict(q=P[0] + 1), INVALID),
    (dict(type=F32, v=P[2] + 2), INVALID), (dict(gq=P[3] + 1), INVALID), (dict(qo=P[0], ldqo=512), INVALID),
    (dict(ko=P[1], ldko=128), INVALID), (dict(qo=P[1]), INVALID), (dict(qo=P[3]), INVALID), (dict(qo=P[6]), INVALID),
    (dict(qo=P[10]), INVALID), (dict(qo=P[8]), INVALID), (dict(kc=P[9]), INVALID), (dict(ko=P[9], ldko=128), INVALID),
    (dict(vc=P[2]), INVALID),
])
def test_qk_refusals(kw, status):
    refused(qk, status, **kw)


def attn(q=P[0], ldq=512, T=4, H=4, Hkv=2, D=128, start=P[1], lens=P[2], B=2, table=P[3], stride=4, kc=P[4], vc=P[5], scale=0.1,
         causal=True, window=0, sink=None, out=P[6], ldo=512, lse=None, ws=P[7], ws_bytes=1 << 30, **kv):
    args = dict(num_blocks=8, block_size=16, block_stride=4096, row_stride=256, head_stride=128)
    args.update(kv)
    dsa.dsa_paged_attn(q, ldq, T, H, Hkv, D, start, lens, B, table, stride, dsa.dsa_kv_cache(kc, vc, *args.values()), scale, causal,
                       window, sink, out, ldo, lse, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(B=65537), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(T=1 << 33), UNSUPPORTED), (dict(window=-1), INVALID), (dict(stride=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID),
    (dict(start=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(out=None), INVALID), (dict(ldq=511), INVALID), (dict(ldo=504), INVALID), (dict(ldq=516), INVALID),
    (dict(ldo=516), INVALID), (dict(row_stride=260), INVALID), (dict(block_stride=4100), INVALID), (dict(head_stride=132), INVALID),
    (dict(q=P[0] + 8), INVALID), (dict(kc=P[4] + 8), INVALID), (dict(vc=P[5] + 2), INVALID), (dict(out=P[6] + 8), INVALID),
    (dict(start=P[1] + 2), INVALID), (dict(sink=P[8] + 2), INVALID), (dict(lse=P[8] + 2), INVALID), (dict(out=P[0]), INVALID),
    (dict(out=P[4]), INVALID), (dict(lse=P[6]), INVALID), (dict(lse=P[2]), INVALID), (dict(ws=P[6]), INVALID), (dict(ws=P[3]), INVALID),
    (dict(num_blocks=0), INVALID), (dict(num_blocks=-1), INVALID), (dict(block_size=0), INVALID), (dict(row_stride=64), INVALID),
    (dict(num_blocks=1 << 30, block_size=64, block_stride=64 * 256), UNSUPPORTED), (dict(block_stride=4096 + 8), UNSUPPORTED),
    (dict(head_stride=256 + 8, Hkv=2), UNSUPPORTED), (dict(ldq=1 << 39), UNSUPPORTED), (dict(row_stride=1 << 39), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=P[7] + 8), WORKSPACE),
])
def test_attn_refusals(kw, status):
    refused(attn, status, **kw)


def test_empty_calls_launch_nothing():
    before = dsa.dsa_launch_count()
    table(n=0)
    rope(T=0)
    rope(H=0)
    qk(T=0)
    qk(H=0, Hkv=0)
    attn(T=0, ws=None, ws_bytes=0)
    attn(B=0, ws=None, ws_bytes=0)
    assert dsa.dsa_launch_count() == before


def test_workspace_sizes():
    ws = dsa.dsa_paged_attn_workspace_bytes
    assert ws(0, 4, 8, 1, 128) == 0 and ws(4, 0, 8, 1, 128) == 0 and ws(4, 4, 8, 3, 128) == 0 and ws(4, 4, 8, 1, 80) == 0
    # two parts of a row block per SM, in fp32: 128 rows where sequences bring few, 256 else
    one, two = ws(64, 64, 64, 8, 128), ws(8192, 1, 64, 8, 128)
    assert 148 * 2 * 128 * 128 * 4 <= one < 32 << 20 and 148 * 2 * 256 * 128 * 4 <= two < 64 << 20
    assert ws(64, 64, 64, 8, 64) < one
    # many sequences: the plan lies there too
    assert ws(20000, 20000, 8, 8, 64) > ws(64, 64, 8, 8, 64) + 20000 * 16


def test_cache_structure_from_tensors():
    torch = pytest.importorskip("torch")
    k, v = (torch.empty(7, 16, 5, 64, dtype=torch.bfloat16) for _ in range(2))
    kv = dsa.make_kv_cache(k, v)
    assert (kv.num_blocks, kv.block_size, kv.block_stride, kv.row_stride, kv.head_stride) == (7, 16, 16 * 320, 320, 64)
    assert kv.k == k.data_ptr() and kv.v == v.data_ptr()
    hm = torch.empty(7, 5, 16, 64, dtype=torch.bfloat16)
    kv = dsa.make_kv_cache(hm.transpose(1, 2))
    assert (kv.block_size, kv.row_stride, kv.head_stride, kv.v) == (16, 64, 1024, None)
    assert dsa.make_kv_cache(None).k is None
    for bad in ((k, v[:, :8]), (k, hm.transpose(1, 2)), (k[..., ::2], v[..., ::2])):
        with pytest.raises(ValueError):
            dsa.make_kv_cache(*bad)


def test_workspace_sizes_of_larger_steps():
    # (only refusals are made here: the addresses are not real)
    ws = dsa.dsa_paged_attn_workspace_bytes
    one, two = ws(300, 300, 64, 8, 128), ws(300, 1, 64, 8, 128)
    assert one < two                                         # a size of its own for one and for two row tiles
    refused(attn, WORKSPACE, T=300, B=1, H=64, Hkv=8, ldq=8192, ldo=8192, row_stride=1024, block_stride=16384,
            ws_bytes=ws(1, 1, 64, 8, 128) - 1)
    # at the same number of tiles the size grows with T and B
    steps = [(t, b) for t in (1, 5, 128, 1000, 20000) for b in (1, 7, 300, 5000)]
    for T, B in steps:
        for T2, B2 in steps:
            same = (T * 8 > 128 * B) == (T2 * 8 > 128 * B2)
            if T <= T2 and B <= B2 and same:
                assert ws(T, B, 64, 8, 128) <= ws(T2, B2, 64, 8, 128)


@pytest.mark.parametrize("amplitude", [1e39, -1e300, 3.5e38])
def test_table_refuses_an_amplitude_past_fp32(amplitude):
    refused(table, INVALID, amplitude=amplitude)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_attn_refuses_a_scale_past_fp32_in_base_2(scale):
    # the softmax multiplies scores by scale log2(e): with an infinite factor a score of zero would be no number
    refused(attn, INVALID, scale=scale)
