"""nc_gemm_fp8 with scales far from 1.  The product of a block's two scales is a
factor in fp32: all bits while it is of normal size, however far apart the two
are; absolute steps of 2^-149 below that; never a finite wrong value above."""
import numpy as np
import pytest

import test_fp8_gpu as base

pytestmark = pytest.mark.gpu
nc = base.nc

SHAPES = [(3, 140, 300), (9, 38400, 300), (50, 300, 400), (200, 300, 1300),   # 16 to 128 rows, K cut or not
          (700, 1300, 700), (4000, 1300, 272),                                # pairs, one tile each and several
          (513, 1100, 3200), (400, 1300, 6416)]                               # pairs, K cut over two and four of them


def _operands(M, N, K, ea, eb):
    """Scales around 2^ea and 2^eb (odd rows': in the middle of fp32's range), and codes as small (or large) as leaves
    sums of normal size."""
    import torch
    g = torch.Generator().manual_seed(M + N + K)
    e8, ld, kb = torch.float8_e4m3fn, -(-K // 16) * 16, base._blocks(K)
    size = 2.0 ** -7 if ea + eb > 0 else 200.0
    a = (torch.randn(M, ld, generator=g) * size).clamp(-448, 448).to(e8)
    b = (torch.randn(N, ld, generator=g) * size).clamp(-448, 448).to(e8)
    b.view(torch.uint8)[::3] = 0          # weight rows of zeros
    a.view(torch.uint8)[M // 2] = 0       # and a row
    sa = torch.exp(0.25 * torch.randn(kb, M, generator=g)) * 2.0 ** ea
    sa[:, 1::2] *= 2.0 ** (-64 if ea + eb > 0 else 64)
    sb = torch.exp(0.25 * torch.randn(base._blocks(N), kb, generator=g)) * 2.0 ** eb
    return dict(a=a, lda=ld, b=b, ldb=ld, M=M, N=N, K=K, lsa=M, lsb=kb, sa=sa, sb=sb)


def _exact(c):
    """sum over K blocks of the scaled sums, and the same of magnitudes, in 64 bits."""
    K = c["K"]
    a, b = (c[k].float().double()[:, :K] for k in "ab")
    acc = mag = 0
    for i, k in enumerate(range(0, K, 128)):
        s = c["sa"][i].double()[:, None] * c["sb"][:, i].double().repeat_interleave(128)[:c["N"]][None]
        p, q = a[:, k:k + 128], b[:, k:k + 128]
        acc, mag = acc + (p @ q.t()) * s, mag + (p.abs() @ q.abs().t()) * s
    return acc, mag


def _run(nc, M, N, K, ea, eb):
    import torch
    c = {k: v.cuda() if torch.is_tensor(v) else v for k, v in _operands(M, N, K, ea, eb).items()}
    acc, mag = _exact(c)
    assert float(acc.abs().max()) < 2.0 ** 127
    D = torch.full((M, -(-N // 4) * 4), 5.0, device="cuda")
    assert base._gemm(nc, c, "STORE_F32", D, D.shape[1]) == 0
    assert nc.nc_ops_status(base._stream(), 60000) == 0
    # 2u a product and 4u a block as elsewhere; half of the smallest step, 2^-150, for each block's addition
    return c, D[:, :N].double(), acc, (128 * 2 + 4 * base._blocks(K)) * base.U * mag + base._blocks(K) * 2.0 ** -150


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ea,eb", [(64, 60), (120, 4), (4, 120), (-60, -62), (-14, -107), (20, -141), (-140, 20)])
def test_scale_products_of_normal_size(nc, M, N, K, ea, eb):
    c, D, acc, tol = _run(nc, M, N, K, ea, eb)
    f = c["sa"][:, :, None].double() * c["sb"].t()[:, None].double()   # 2^(+-2.5) around 2^(ea + eb) and odd rows'
    assert 2.0 ** -126 <= float(f.min()) and float(f.max()) < 2.0 ** 128
    assert bool(((D - acc).abs() <= tol).all())
    assert bool((D[:, ::3] == 0).all()) and bool((D[M // 2] == 0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ea,eb", [(-80, -63), (-30, -113), (-149, -149)])
def test_scale_products_below_normal_size(nc, M, N, K, ea, eb):
    """A factor is off by at most half a step, 2^-150, which counts times the block's sum of codes."""
    import torch
    c, D, acc, tol = _run(nc, M, N, K, ea, eb)
    codes = c["a"].float().double()[:, :K].abs() @ c["b"].float().double()[:, :K].abs().t()
    assert bool(((D - acc).abs() <= tol + codes * 2.0 ** -150).all())
    assert bool((D[:, ::3] == 0).all()) and bool((D[M // 2] == 0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ea,eb", [(70, 62), (122, 10)])
def test_scale_products_above_the_range_are_not_finite(nc, M, N, K, ea, eb):
    import torch
    c = {k: v.cuda() if torch.is_tensor(v) else v for k, v in _operands(M, N, K, ea, eb).items()}
    D = torch.zeros(M, -(-N // 4) * 4, device="cuda")
    assert base._gemm(nc, c, "STORE_F32", D, D.shape[1]) == 0
    assert nc.nc_ops_status(base._stream(), 60000) == 0
    f = c["sa"][:, ::2, None].double() * c["sb"].t()[:, None].double()  # the even rows'
    assert float(f.min()) > 2.0 ** 128
    assert not bool(torch.isfinite(D[::2, :N]).any())
    assert bool(torch.isfinite(D[1::2, :N]).all())
