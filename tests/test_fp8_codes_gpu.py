"""The 8-bit output of nc_gemm_fp8 (NC_EPI_RELU2_FP8): its codes and scales are
those that the definition gives for the call's own fp32 sums,
RN_e4m3(RN(RN(448 v) / a)) of v = RN(relu(acc)^2) and RN(a / 448), bit for bit."""
import numpy as np
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc  # the module's fixture

# M, N, K: every kernel and way of cutting K
SHAPES = [
    (1, 300, 16), (9, 38400, 16), (30, 1003, 400), (60, 300, 1300), (200, 300, 1300),   # 16 to 128 rows, K cut or not
    (700, 1300, 144), (300, 2000, 48),        # pairs of CTAs
    (513, 1100, 3200), (400, 1300, 6416),     # pairs, K cut over two and four of them
]


def _one_product(M, N, K, x, b):
    """Operands whose sums are RN(x[m] b[n]) exactly: one product of codes 1 and b, scaled by x."""
    import torch
    e8 = torch.float8_e4m3fn
    ld = -(-K // 16) * 16
    a = torch.zeros(M, ld, device="cuda")
    a[:, 0] = 1
    w = torch.zeros(N, ld, device="cuda")
    w[:, 0] = torch.from_numpy(b).cuda()
    kb = base._blocks(K)
    sa = torch.ones(kb, M, device="cuda")
    sa[0] = torch.from_numpy(x).cuda()
    return dict(a=a.to(e8), lda=ld, sa=sa, lsa=M, b=w.to(e8), ldb=ld, sb=torch.ones(base._blocks(N), kb, device="cuda"),
                lsb=kb, M=M, N=N, K=K)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_codes_of_exact_sums(nc, M, N, K):
    """Sums known exactly, among them ties: (x / (256 x))^2 448 = 7 2^-10 lies halfway between two codes."""
    import torch
    r = np.random.RandomState(M + N)
    x = (r.uniform(1, 2, M) * 2.0 ** r.randint(-72, 50, M)).astype(np.float32)
    values = np.arange(128, dtype=np.uint8)[:0x79]      # the codes 0 .. 256 (0x78)
    values = torch.from_numpy(values).view(torch.float8_e4m3fn).float().numpy()
    b = r.choice(values, N).astype(np.float32)
    b[::5] = 1
    b[3::7] *= -1
    b[::128] = 256                                      # the largest of every block
    c = _one_product(M, N, K, x, b)
    ldd = -(-N // 16) * 16
    q = torch.zeros(M, ldd, device="cuda").to(torch.float8_e4m3fn)
    sd = torch.empty(base._blocks(N), M, device="cuda")
    assert base._gemm(nc, c, "RELU2_FP8", q, ldd, sd, M) == 0
    assert nc.nc_ops_status(base._stream(), 60000) == 0
    acc = np.maximum(x[:, None] * b[None], np.float32(0))
    v = acc * acc
    a = base._block_max(v, 1).astype(np.float32)        # exact: a maximum
    ax = base._expand(a, M, N, 1).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(ax > 0, (np.float32(448) * v) / ax, np.float32(0))
    np.testing.assert_array_equal(base._host(q)[:, :N], base._e4m3(z))
    np.testing.assert_array_equal(sd.cpu().numpy(), a / np.float32(448))


@pytest.mark.parametrize("M,N,K", SHAPES + [(4096, 5120, 272)])
def test_fused_codes_are_the_quantisers(nc, M, N, K):
    """Fused, and as fp32 sums, their squares and the quantiser: the same bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M * 3 + N)
    e8 = torch.float8_e4m3fn
    ld, kb, nb = -(-K // 16) * 16, base._blocks(K), base._blocks(N)

    def rand(*n):
        return torch.randn(*n, device="cuda", generator=g)
    c = dict(a=(rand(M, ld) * 60).clamp(-448, 448).to(e8), lda=ld, sa=torch.exp(rand(kb, M)), lsa=M,
             b=(rand(N, ld) * 60).clamp(-448, 448).to(e8), ldb=ld, sb=torch.exp(rand(nb, kb)) * 1e-3, lsb=kb, M=M, N=N, K=K)
    N16 = -(-N // 16) * 16                              # the quantiser takes whole sixteens: the rest is zeros
    acc = torch.zeros(M, N16, device="cuda")
    q, want = (torch.zeros(M, N16, device="cuda").to(e8) for _ in range(2))
    sd, sw = (torch.empty(nb, M, device="cuda") for _ in range(2))
    assert base._gemm(nc, c, "RELU2_FP8", q, N16, sd, M) == 0
    assert base._gemm(nc, c, "STORE_F32", acc, N16) == 0
    v = torch.relu(acc).square()
    assert nc.nc_quant_fp8(v.data_ptr(), N16, want.data_ptr(), N16, sw.data_ptr(), M, M, N16, 1, nc.NC_F32,
                           base._stream()) == 0
    assert nc.nc_ops_status(base._stream(), 60000) == 0
    assert (v > 0).any()
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(sd, sw)
