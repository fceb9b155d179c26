"""Each 8-bit call reads what the call right before it in the stream wrote, without a wait on the host between
(the kernels may start while the one before them still runs): the bits are those of the same calls waited for."""
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 300, 4100])
def test_quantisers_behind_norm_and_product(nc, dtype, M):
    """norm -> both quantisers of its x_out -> a product of the codes onto that same x_out (bf16) -> the next round."""
    import torch
    C, n, e8 = 640, 30, torch.float8_e4m3fn
    kb = C // 128
    g = torch.Generator(device="cuda").manual_seed(M)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    code = nc.NC_BF16 if dtype == "bf16" else nc.NC_F32
    x0 = torch.randn(M, C, device="cuda", generator=g).to(t)
    res = [torch.randn(M, C, device="cuda", generator=g).to(t) for _ in range(3)]
    w = torch.randn(C, C, device="cuda", generator=g).to(t)
    x, wq, q, q2 = x0.clone(), torch.empty(C, C, device="cuda").to(e8), x0.to(e8), x0.to(e8)
    d = torch.zeros(M, C, device="cuda", dtype=torch.bfloat16)
    s, s2 = torch.empty(kb, M, device="cuda"), torch.empty(-(-M // 128), kb, device="cuda")
    sw = torch.empty(kb, kb, device="cuda")

    def run(wait):
        st = base._stream()
        keep = []

        def call(rc):
            assert rc == 0
            if wait:
                torch.cuda.synchronize()
        x.copy_(x0)
        d.zero_()
        for i in range(n):
            call(nc.nc_add_rmsnorm_fp8(x.data_ptr(), res[i % 3].data_ptr(), x.data_ptr(), q.data_ptr(), s.data_ptr(), M,
                                       None, M, C, code, st))
            call(nc.nc_quant_fp8(x.data_ptr(), C, q2.data_ptr(), C, s2.data_ptr(), kb, M, C, 128, code, st))
            call(nc.nc_quant_fp8(x.data_ptr(), C, q.data_ptr(), C, s.data_ptr(), M, M, C, 1, code, st))
            call(nc.nc_quant_fp8(w.data_ptr(), C, wq.data_ptr(), C, sw.data_ptr(), kb, C, C, 128, code, st))
            call(nc.nc_gemm_fp8(q.data_ptr(), C, s.data_ptr(), M, wq.data_ptr(), C, sw.data_ptr(), kb, d.data_ptr(), C, None,
                                0, M, C, C, nc.NC_EPI_STORE, st))
            call(nc.nc_quant_fp8(d.data_ptr(), C, q.data_ptr(), C, s.data_ptr(), M, M, C, 1, nc.NC_BF16, st))
            if i % 7 == 6:
                keep += [a.clone() for a in (x, q.view(torch.uint8), s, q2.view(torch.uint8), s2, d)]
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return keep + [a.clone() for a in (x, q.view(torch.uint8), s, q2.view(torch.uint8), s2, d)]
    want = run(True)
    assert all(torch.isfinite(a.float()).all() for a in want)
    for _ in range(4):
        for a, b in zip(want, run(False)):
            assert torch.equal(a, b)
    assert nc.nc_ops_status(base._stream(), 60000) == 0
