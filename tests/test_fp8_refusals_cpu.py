"""Sizes whose grids no launch can hold are refused as shapes, before any CUDA call."""
import pytest

import decoder_only_transformer_nanochat_b200 as nc
from decoder_only_transformer_nanochat_b200 import build as nc_build

BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    nc_build.build()
    return nc.load_library()


@pytest.mark.parametrize("rows,cols,block_rows", [(2 ** 31 - 1, BIG, 1), (2 ** 31 - 1, 8208, 1), (2 ** 31 - 1, BIG, 128),
                                                  (2 ** 31 - 1, 16400, 128)])
def test_quant_beyond_a_grid(rows, cols, block_rows):
    pieces = -(-rows // (32 if block_rows == 1 else 128)) * -(-cols // (256 if block_rows == 1 else 128))
    assert pieces > 2 ** 31 - 1
    assert nc.nc_quant_fp8(16, cols, 16, cols, 16, 2 ** 31, rows, cols, block_rows, nc.NC_BF16, None) == nc.NC_ESHAPE


@pytest.mark.parametrize("M,N", [(BIG, BIG), (BIG, 16385), (16385, BIG), (2 ** 22 + 1, 2 ** 22)])
def test_gemm_beyond_a_grid(M, N):
    assert -(-M // 128) * -(-N // 128) > 2 ** 30
    for epi in (nc.NC_EPI_STORE, nc.NC_EPI_RELU2_FP8):
        assert nc.nc_gemm_fp8(16, 128, 16, M, 16, 128, 16, 1, 16, -(-N // 16) * 16, 16, M, M, N, 128, epi, None) == nc.NC_ESHAPE


@pytest.mark.parametrize("dtype", [-1, 2, 7])
def test_other_types(dtype):
    assert nc.nc_add_rmsnorm_fp8(16, 16, 16, 16, 16, 8, 16, 8, 128, dtype, None) == nc.NC_EUNSUPPORTED
    assert nc.nc_quant_fp8(16, 256, 16, 256, 16, 8, 8, 256, 1, dtype, None) == nc.NC_EUNSUPPORTED
