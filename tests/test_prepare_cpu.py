"""Host side of the calls that prepare a step's inputs, without a GPU: refusals before any
launch, and the tests' plain references pinned to hand-worked cases."""
import numpy as np
import pytest

import prepare_ref as ref
from test_abi_cpu import FAKE, _status, lib  # noqa: F401  (lib: the built library)
from deepseek_v4_sparse_dsa_gb300 import dsa

INVALID, UNSUPPORTED = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED


def _p(i):
    return FAKE + (i << 16)


def slots(cached=_p(1), new=_p(2), B=4, bs=64, free=_p(3), n_free=8, nblk=100, table=_p(4), stride=8, tokens=16,
          ctx=_p(5), start=_p(6), slot=_p(7), pos=_p(8), used=_p(9)):
    return _status(dsa.dsa_assign_slots, cached, new, B, bs, free, n_free, nblk, table, stride, tokens, ctx, start,
                   slot, pos, used, 0)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(bs=0), INVALID), (dict(n_free=-1), INVALID), (dict(nblk=-1), INVALID),
    (dict(tokens=-1), INVALID), (dict(stride=0), INVALID), (dict(B=65537), UNSUPPORTED), (dict(tokens=2**31), UNSUPPORTED),
    (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(free=None), INVALID), (dict(table=None), INVALID),
    (dict(ctx=None), INVALID), (dict(start=None), INVALID), (dict(slot=None), INVALID), (dict(pos=None), INVALID),
    (dict(used=None), INVALID), (dict(cached=_p(1) + 2), INVALID), (dict(slot=_p(7) + 4), INVALID),
    (dict(ctx=_p(1)), INVALID), (dict(ctx=_p(2)), INVALID), (dict(table=_p(3)), INVALID), (dict(pos=_p(7)), INVALID),
])
def test_assign_slots_refusals(lib, bad, status):  # noqa: F811
    before = dsa.dsa_launch_count()
    assert slots(**bad) == status
    assert dsa.dsa_launch_count() == before


def norm(x=_p(1), ldx=256, res=_p(2), ldr=256, gamma=_p(3), eps=1e-6, T=4, D=256, typ=dsa.DSA_REAL_BF16, ro=_p(4),
         y=_p(5), codes=_p(6), ldy=256, scale=_p(7), pow2=False):
    return _status(dsa.dsa_add_rmsnorm_e4m3, x, ldx, res, ldr, gamma, eps, T, D, typ, ro, y, codes, ldy, scale, pow2, 0)


@pytest.mark.parametrize("bad,status", [
    (dict(typ=2), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(D=32769), UNSUPPORTED),
    (dict(T=2**31), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(gamma=None), INVALID), (dict(ldx=255), INVALID),
    (dict(ldr=255), INVALID), (dict(res=None, ldr=255), INVALID), (dict(ldy=255), INVALID), (dict(scale=None), INVALID),
    (dict(codes=None), INVALID), (dict(ro=None, y=None, codes=None, scale=None), INVALID), (dict(x=_p(1) + 1), INVALID),
    (dict(typ=dsa.DSA_REAL_F32, x=_p(1) + 2), INVALID), (dict(scale=_p(7) + 2), INVALID),
    (dict(ro=_p(1), ldx=264), INVALID), (dict(y=_p(1), ldx=264), INVALID), (dict(y=_p(2)), INVALID),
    (dict(y=_p(4)), INVALID), (dict(codes=_p(1)), INVALID), (dict(codes=_p(2)), INVALID), (dict(codes=_p(5)), INVALID),
])
def test_add_rmsnorm_refusals(lib, bad, status):  # noqa: F811
    before = dsa.dsa_launch_count()
    assert norm(**bad) == status
    assert dsa.dsa_launch_count() == before


@pytest.mark.parametrize("bad", [dict(scale=_p(1)), dict(scale=_p(2)), dict(scale=_p(3)), dict(scale=_p(4)), dict(scale=_p(5)),
                                 dict(scale=_p(6)), dict(gamma=_p(4)), dict(gamma=_p(5)), dict(gamma=_p(6))])
def test_add_rmsnorm_refuses_outputs_at_gamma_and_anything_at_the_scales(lib, bad):  # noqa: F811
    # every row reads gamma and no other row's scales: an output there would change later rows
    before = dsa.dsa_launch_count()
    assert norm(**bad) == INVALID
    assert dsa.dsa_launch_count() == before


def gemm(a=_p(1), lda=256, asc=_p(2), w=_p(3), ldw=256, wsc=_p(4), M=4, N=128, K=256, out=_p(5), ldo=128,
         typ=dsa.DSA_REAL_BF16):
    return _status(dsa.dsa_gemm_e4m3, a, lda, asc, w, ldw, wsc, M, N, K, out, ldo, typ, 0)


@pytest.mark.parametrize("bad,status", [
    (dict(typ=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID),
    (dict(M=2**31), UNSUPPORTED), (dict(a=None), INVALID), (dict(asc=None), INVALID), (dict(w=None), INVALID),
    (dict(wsc=None), INVALID), (dict(out=None), INVALID), (dict(lda=240), INVALID), (dict(ldw=240), INVALID),
    (dict(lda=264), INVALID), (dict(ldw=264), INVALID), (dict(ldo=127), INVALID), (dict(a=_p(1) + 8), INVALID),
    (dict(w=_p(3) + 8), INVALID), (dict(out=_p(5) + 1), INVALID), (dict(out=_p(5) + 2, typ=dsa.DSA_REAL_F32), INVALID),
    (dict(asc=_p(2) + 1), INVALID), (dict(out=_p(1)), INVALID), (dict(out=_p(3)), INVALID), (dict(lda=1 << 40), UNSUPPORTED), (dict(ldw=1 << 40), UNSUPPORTED),
    (dict(M=2**31 - 300, N=2**31 - 300, ldo=2**31), UNSUPPORTED),
])
def test_gemm_refusals(lib, bad, status):  # noqa: F811
    before = dsa.dsa_launch_count()
    assert gemm(**bad) == status
    assert dsa.dsa_launch_count() == before


def test_empty_problems_are_no_ops(lib):  # noqa: F811
    before = dsa.dsa_launch_count()
    assert norm(x=None, gamma=None, T=0, codes=None, scale=None, y=None, ro=None) == dsa.DSA_OK
    assert gemm(a=None, asc=None, w=None, wsc=None, out=None, M=0) == dsa.DSA_OK
    assert gemm(a=None, asc=None, w=None, wsc=None, out=None, N=0) == dsa.DSA_OK
    assert dsa.dsa_launch_count() == before


@pytest.mark.parametrize("bad", [3.9, 4096.0, "128", b"128", np.int64(4096), np.array(4096), np.array([4096]), [4096]])
def test_only_integers_and_tensors_are_addresses(lib, bad):  # noqa: F811
    # whatever int() would make an address of is refused before the call, for every argument that is one
    before = dsa.dsa_launch_count()
    for call in (lambda: slots(cached=bad), lambda: norm(gamma=bad), lambda: gemm(w=bad),
                 lambda: _status(dsa.dsa_indexer_k_hadamard_mxfp4, bad, _p(1), 0, 128, _p(2), _p(3), 64, 0)):
        with pytest.raises((AttributeError, TypeError)):
            call()
    assert dsa.dsa_launch_count() == before
    assert dsa._ptr(4096) == 4096 and dsa._ptr(None) is None


# ------------------------------------------------------------------ the references
def test_reference_slots_by_hand():
    # block size 4; request 0 holds 3 tokens (1 page) and brings 3: one slot left in page 7, then a new page;
    # request 1 brings nothing; request 2 holds 4 (a full page) and brings 1: a new page
    table = np.array([[7, -1, -1], [5, -1, -1], [2, -1, -1]])
    t, ctx, start, slot, pos, used = ref.assign_slots(np.array([3, 2, 4]), np.array([3, 0, 1]), 4, [9, 0, 8], 10, table, 6)
    assert t.tolist() == [[7, 9, -1], [5, -1, -1], [2, 0, -1]]
    assert ctx.tolist() == [6, 2, 5] and start.tolist() == [0, 3, 3, 4] and used == 2
    assert slot.tolist() == [31, 36, 37, 0, -1, -1] and pos.tolist() == [3, 4, 5, 4, 0, 0]


def test_reference_norm_by_hand():
    r, y = ref.add_rmsnorm([[3.0, 0.0]], [[0.0, 4.0]], [1.0, 2.0], 1e-12, True)
    assert r.tolist() == [[3.0, 4.0]]
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    # 1 + 2^-8 is a tie between 1 and 1 + 2^-7: to the even one; just above goes up
    assert ref.bf16_round([1 + 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -20]).tolist() == [1.0, 1 + 2.0 ** -7]


def test_reference_values_and_gemm_by_hand():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(ref.e4m3_values(), t, equal_nan=True)
    # 129 ones per row: block 0 holds 128 of them, block 1 one
    a, w = np.full((1, 129), 0x38, np.uint8), np.full((2, 129), 0x38, np.uint8)
    out, _ = ref.gemm(a, np.array([[2.0, 3.0]]), w, np.array([[0.5, 10.0]]))
    assert out.tolist() == [[128 * 1.0 + 30.0] * 2]
