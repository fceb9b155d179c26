"""The softcap of nc_gemm_fp8 keeps its relative accuracy down to the smallest sums."""
import numpy as np
import pytest

import test_fp8_gpu as base
from test_fp8_codes_gpu import _one_product

pytestmark = pytest.mark.gpu
nc = base.nc


@pytest.mark.parametrize("M,N,K", [(13, 300, 16), (9, 38400, 16), (200, 300, 1300), (700, 1300, 144), (513, 1100, 3200)])
def test_softcap_of_exact_sums(nc, M, N, K):
    """Sums RN(x b) known exactly, from 2^-40 to beyond the cap.  15 tanh(z / 15) in fp32: z itself below 0.09 leaves
    (z / 15)^2 / 3 < 2^-16.3 out; from there on E is off by at most 2^-22 (2^-22.5 of the exponential, half a unit of its
    argument's scaling), which 1 - E >= 2^-6.4 turns into 2^-15.6, and sum and quotient add 2^-21.8: below 2^-15.5
    together.  bf16 adds half a step."""
    import torch
    r = np.random.RandomState(N)
    x = (r.uniform(1, 2, M) * 2.0 ** r.randint(-40, 4, M)).astype(np.float32)
    b = r.choice(np.array([0, 0.125, 0.5, 1, 1.5, 2, 3.25, 7, -1, -0.875, -4], np.float32), N)
    c = _one_product(M, N, K, x, b)
    D = torch.zeros(M, -(-N // 8) * 8, device="cuda", dtype=torch.bfloat16)
    assert base._gemm(nc, c, "SOFTCAP", D, D.shape[1]) == 0
    assert nc.nc_ops_status(base._stream(), 60000) == 0
    ref = 15 * np.tanh((x[:, None] * b[None]).astype(np.float64) / 15)
    err = np.abs(base._host(D)[:, :N] - ref)
    assert (err <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -15)).all(), np.nanmax(err / np.maximum(np.abs(ref), 1e-300))
