"""The counted wait of the 8-bit GEMM runs out and reaches the host (through the library's self-check)."""
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc


@pytest.mark.parametrize("wait_us", [0, 1000, 100000])
def test_expired_counted_wait(nc, wait_us):
    import torch
    st = base._stream()
    assert nc.nc_ops_status(st, 60000) == nc.NC_OK
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    assert nc.nc_check_wait_expiry(wait_us, st) == nc.NC_OK
    b.record()
    assert nc.nc_ops_status(st, 60000) == nc.NC_ETIMEOUT
    assert nc.nc_ops_status(st, 60000) == nc.NC_OK
    # the wait limited by the clock, then wait_us / 4 tries and up to 256 more before the next look at the limit: well above
    # the first alone if a try takes anything near its 4 us
    us = 1000 * a.elapsed_time(b)
    print(f"wait_us {wait_us}: {us:.0f} us")
    assert us >= 1.5 * wait_us
    # the context and the GEMM are as before
    c = base._case(nc, 300, 520, 400)
    base._check(nc, c, "STORE")
