"""8-bit calls behind a join of streams: a product waits for its activations and, through an event, for the weights that
another stream quantises; eager and captured into a graph."""
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc


@pytest.mark.parametrize("M,C,N", [(3, 640, 1300), (300, 1504, 900), (5000, 640, 2000)])
def test_product_behind_a_join(nc, M, C, N):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    e8 = torch.float8_e4m3fn
    kb, nb = base._blocks(C), base._blocks(N)
    x, w = (torch.randn(r, C, device="cuda", generator=g).bfloat16() for r in (M, N))
    ldd = -(-N // 16) * 16
    b = dict(q=x.to(e8), s=torch.empty(kb, M, device="cuda"), wq=w.to(e8), sw=torch.empty(nb, kb, device="cuda"),
             d=torch.zeros(M, ldd, device="cuda").bfloat16(), h=torch.zeros(M, ldd, device="cuda").to(e8),
             sh=torch.empty(nb, M, device="cuda"))
    side = torch.cuda.Stream()

    def clear():
        for k in ("q", "wq", "h"):
            b[k].view(torch.uint8).zero_()
        for k in ("s", "sw", "d", "sh"):
            b[k].zero_()

    def run(join=True):
        main = torch.cuda.current_stream()
        fork = torch.cuda.Event()
        fork.record(main)
        other = side if join else main
        other.wait_event(fork)
        assert nc.nc_quant_fp8(w.data_ptr(), C, b["wq"].data_ptr(), C, b["sw"].data_ptr(), kb, N, C, 128, nc.NC_BF16,
                               other.cuda_stream) == 0
        done = torch.cuda.Event()
        done.record(other)
        assert nc.nc_add_rmsnorm_fp8(x.data_ptr(), None, x.data_ptr(), b["q"].data_ptr(), b["s"].data_ptr(), M, None, M, C,
                                     nc.NC_BF16, main.cuda_stream) == 0
        main.wait_event(done)
        for epi, D, sd in (("STORE", b["d"], None), ("RELU2_FP8", b["h"], b["sh"])):
            assert nc.nc_gemm_fp8(b["q"].data_ptr(), C, b["s"].data_ptr(), M, b["wq"].data_ptr(), C, b["sw"].data_ptr(), kb,
                                  D.data_ptr(), ldd, sd.data_ptr() if sd is not None else None, M, M, N, C,
                                  getattr(nc, "NC_EPI_" + epi), main.cuda_stream) == 0

    def outputs():
        torch.cuda.synchronize()
        return b["d"].clone(), b["h"].view(torch.uint8).clone(), b["sh"].clone()
    clear()
    torch.cuda.synchronize()
    run(join=False)
    want = outputs()
    assert (want[0] != 0).any()
    for _ in range(5):
        clear()
        torch.cuda.synchronize()
        run()
        assert all(torch.equal(a, c) for a, c in zip(want, outputs()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        clear()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(want, outputs()))
    assert nc.nc_ops_status(base._stream(), 60000) == 0
