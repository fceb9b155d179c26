"""The 8-bit entry points' argument checks (host only: each call below returns
before any device work or CUDA call)."""
import pytest

import decoder_only_transformer_nanochat_b200 as nc
from decoder_only_transformer_nanochat_b200 import build as nc_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    nc_build.build()
    return nc.load_library()


def _norm(x=16, res=16, x_out=16, q=16, s=16, lds=8, r=16, M=8, C=128, dtype=nc.NC_BF16):
    return nc.nc_add_rmsnorm_fp8(x, res, x_out, q, s, lds, r, M, C, dtype, None)


def test_add_rmsnorm_refusals():
    for name in ("x", "x_out", "q", "s"):
        assert _norm(**{name: None}) == nc.NC_EINVAL, name
    for bad in (dict(M=0), dict(M=-1), dict(C=0), dict(C=8), dict(C=120), dict(C=4112), dict(lds=7)):
        assert _norm(**bad) == nc.NC_ESHAPE, bad
    for name in ("x", "res", "x_out", "q"):
        assert _norm(**{name: 24}) == nc.NC_EALIGN, name
    for name in ("s", "r"):
        assert _norm(**{name: 18}) == nc.NC_EALIGN, name
    assert _norm(dtype=2) == nc.NC_EUNSUPPORTED


def _quant(x=16, ldx=256, q=16, ldq=256, s=16, lds=8, rows=8, cols=256, block_rows=1, dtype=nc.NC_BF16):
    return nc.nc_quant_fp8(x, ldx, q, ldq, s, lds, rows, cols, block_rows, dtype, None)


def test_quant_refusals():
    for name in ("x", "q", "s"):
        assert _quant(**{name: None}) == nc.NC_EINVAL, name
    for b in (0, 2, 64, 129):
        assert _quant(block_rows=b) == nc.NC_EINVAL
    for bad in (dict(rows=0), dict(cols=0), dict(cols=8), dict(cols=250), dict(ldx=248), dict(ldq=240), dict(lds=7),
                dict(block_rows=128, lds=1), dict(cols=(1 << 30) + 16, ldx=1 << 31, ldq=1 << 31)):
        assert _quant(**bad) == nc.NC_ESHAPE, bad
    for bad in (dict(x=24), dict(q=20), dict(s=17), dict(ldx=260), dict(ldq=264), dict(dtype=nc.NC_F32, ldx=258)):
        assert _quant(**bad) == nc.NC_EALIGN, bad
    assert _quant(dtype=5) == nc.NC_EUNSUPPORTED


def _gemm(A=16, lda=256, sa=16, lsa=8, B=16, ldb=256, sb=16, lsb=2, D=16, ldd=64, sd=16, lsd=8, M=8, N=64, K=256,
          epi=nc.NC_EPI_STORE):
    return nc.nc_gemm_fp8(A, lda, sa, lsa, B, ldb, sb, lsb, D, ldd, sd, lsd, M, N, K, epi, None)


def test_gemm_refusals():
    for name in ("A", "sa", "B", "sb", "D"):
        assert _gemm(**{name: None}) == nc.NC_EINVAL, name
    # no such epilogue here: the relu^2 backward and the accumulation belong to training
    for epi in (nc.NC_EPI_DRELU2, 6, 8, -1):
        assert _gemm(epi=epi) == nc.NC_EINVAL
    assert _gemm(epi=nc.NC_EPI_RELU2_FP8, sd=None) == nc.NC_EINVAL
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(M=-4), dict(lda=240), dict(ldb=240), dict(ldd=56), dict(lsa=7),
                dict(lsb=1), dict(epi=nc.NC_EPI_RELU2_FP8, lsd=7), dict(M=(1 << 30) + 1, lsa=1 << 31), dict(lda=1 << 38), dict(ldd=1 << 38)):
        assert _gemm(**bad) == nc.NC_ESHAPE, bad
    for bad in (dict(A=24), dict(B=8), dict(D=24), dict(sa=18), dict(sb=17), dict(lda=264), dict(ldb=257), dict(ldd=68),
                dict(epi=nc.NC_EPI_STORE_F32, ldd=66), dict(epi=nc.NC_EPI_RELU2_FP8, ldd=72),
                dict(epi=nc.NC_EPI_RELU2_FP8, sd=18)):
        assert _gemm(**bad) == nc.NC_EALIGN, bad
