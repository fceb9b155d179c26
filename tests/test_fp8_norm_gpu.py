"""nc_add_rmsnorm_fp8 in both of its forms, a warp a row (bf16, 2048 rows or more, up to 2048 wide) and four: sums, codes,
scales and the norm against the definition in 64 bits."""
import numpy as np
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc


def _squares_bound(C, warps):
    """Roundings of a sum of C squares: a lane's 8 ceil(C / (256 warps)) squares one after the other (the square itself one
    more), five levels over a warp, then the warps' sums one after the other."""
    return 8 * -(-C // (256 * warps)) + 1 + 5 + (warps if warps > 1 else 0)


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("C", [16, 208, 256, 272, 640, 784, 1040, 1280, 1536, 1680, 1808, 2048, 2064])
@pytest.mark.parametrize("M,dtype", [(2051, "bf16"), (2047, "bf16"), (2051, "f32"), (4099, "bf16")])
def test_many_rows(nc, M, dtype, C, res):
    import torch
    code = nc.NC_BF16 if dtype == "bf16" else nc.NC_F32
    xd, xv = base._dev(base._rows(C + M, M, C), dtype)
    rd, rv = base._dev(base._rows(C + 1, M, C) * 0.3, dtype)
    want = base._dev(xv + rv, dtype)[1] if res else xv
    lds = M + 3
    xo = torch.full((M + 1, C), 7.0, device="cuda", dtype=xd.dtype)
    q = torch.full((M + 1, C), 3.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((base._blocks(C), lds), -1.0, device="cuda")
    r = torch.full((M + 1,), -1.0, device="cuda")
    assert nc.nc_add_rmsnorm_fp8(xd.data_ptr(), rd.data_ptr() if res else None, xo.data_ptr(), q.data_ptr(),
                                 s.data_ptr(), lds, r.data_ptr(), M, C, code, base._stream()) == 0
    np.testing.assert_array_equal(base._host(xo)[:M], want)
    np.testing.assert_array_equal(base._host(q)[:M], base._codes(want, 1, dtype)[0])
    # nothing behind the last row, nothing between the rows of scales
    assert (xo[M] == 7).all() and (q[M].float() == 3).all() and r[M] == -1 and (s[:, M:] == -1).all()
    r_ref = 1 / np.sqrt((want * want).mean(1) + base.EPS)
    warps = 1 if dtype == "bf16" and M >= 2048 and C <= 2048 else 4
    # half of the sum's, the mean's and eps' roundings (the root halves them), two units of the root
    tol = ((_squares_bound(C, warps) + 2) / 2 + 4) * base.U
    np.testing.assert_allclose(base._host(r)[:M], r_ref, rtol=tol)
    s_ref = base._block_max(want, 1) * r_ref / 448
    np.testing.assert_allclose(base._host(s)[:, :M], s_ref, rtol=tol + 2.01 * base.U)   # its product and quotient


@pytest.mark.parametrize("C", [256, 1280])
def test_special_rows_among_many(nc, C):
    """Rows of zeros, with zero blocks, NaN, infinities and values far below eps, a warp a row."""
    import torch
    M = 2050
    x = base._rows(1, M, C)
    x[0] = 0
    x[7, 128:] = 0
    x[8, 130] = np.nan
    x[9, 5] = np.inf
    x[2049] = 1e-30
    xd, xv = base._dev(x, "bf16")
    q = torch.zeros(M, C, device="cuda").to(torch.float8_e4m3fn)
    s, r = torch.empty(base._blocks(C), M, device="cuda"), torch.empty(M, device="cuda")
    assert nc.nc_add_rmsnorm_fp8(xd.data_ptr(), None, xd.data_ptr(), q.data_ptr(), s.data_ptr(), M, r.data_ptr(), M, C,
                                 nc.NC_BF16, base._stream()) == 0
    with np.errstate(invalid="ignore"):
        y = base._host(q) * base._expand(base._host(s), M, C, 1)
    assert (y[0] == 0).all() and (y[7, 128:] == 0).all()
    assert np.isnan(y[8]).all() and np.isnan(y[9, :128]).all()
    with np.errstate(all="ignore"):
        ref = xv / np.sqrt((xv * xv).mean(1) + base.EPS)[:, None]
    for m in [1, 6, 7, 10, 2048, 2049]:
        step = np.repeat(np.abs(ref[m]).reshape(-1, 128).max(1), 128) / 448
        assert (np.abs(y[m] - ref[m]) <= 2.0 ** -4 * np.abs(ref[m]) + 2.0 ** -10 * step + 1e-5 * np.abs(ref[m])).all(), m
