"""The 8-bit operators (nc_add_rmsnorm_fp8, nc_quant_fp8, nc_gemm_fp8) against
their definitions in 64 bits.

Codes of bf16 inputs are compared exactly: round-to-nearest-even of the exact
quotient 448 v / a (float64 holds it far more closely than the 2^-13 that
separates it from a rounding border it does not sit on).

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  * the norm's sum of squares: a lane adds 8 ceil(C / 256) squares (each
    rounded), then 5 levels over the warp; mean, eps and 1/sqrt (2 units) follow, and the root
    halves the sum's error;
  * one K block on the tensor cores: exact products, 128 additions that
    round or truncate to 24 bits (2u each) of sums no larger than the sum of
    magnitudes; then one rounded multiply-add per block (scale product,
    multiply-add: 2u each block's value, u each running sum);
  * a bf16 output adds half a step, 2^-8 relative; an e4m3 one 2^-4, or half
    its smallest step (2^-10 scale);
  * relu^2 turns an error e of acc into at most 2 |acc| e + e^2; the softcap's
    slope is at most 1 and its exponential formula adds below 15 2^-19.
"""
import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 2.0 ** -23


@pytest.fixture(scope="module")
def nc():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decoder_only_transformer_nanochat_b200 import build
    build.build()
    import decoder_only_transformer_nanochat_b200 as m
    return m


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _dev(a, dtype):
    """(device tensor, the values it holds as fp64)."""
    import torch
    if dtype == "bf16":
        bits = synth.f32_to_bf16_bits(np.ascontiguousarray(a, dtype=np.float32))
        return torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16), synth.bf16_bits_to_f64(bits)
    f = np.ascontiguousarray(a, dtype=np.float32)
    return torch.from_numpy(f.copy()).cuda(), f.astype(np.float64)


def _host(t):
    import torch
    if t.dtype == torch.float8_e4m3fn:
        t = t.float()  # exact
    return t.float().cpu().numpy().astype(np.float64)


def _e4m3(z):
    """fp64 to the nearest e4m3 value, ties to even (|z| <= 448)."""
    z = np.asarray(z, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -30)))
    step = np.exp2(np.maximum(e, -6) - 3)
    return np.rint(z / step) * step


def _blocks(n):
    return -(-n // 128)


def _expand(s, R, K, rows):
    """Scales to one per value."""
    if rows == 1:
        return np.repeat(s.T, 128, 1)[:R, :K]
    return np.repeat(np.repeat(s, 128, 0), 128, 1)[:R, :K]


def _block_max(v, rows):
    R, K = v.shape
    p = np.zeros((-(-R // rows) * rows, _blocks(K) * 128))
    p[:R, :K] = np.abs(v)
    a = p.reshape(-1, rows, _blocks(K), 128).max((1, 3))
    return a.T if rows == 1 else a


def _codes(v, rows, dtype="bf16"):
    """(codes as values, scales) by the definition."""
    a = _block_max(v, rows)
    ax = _expand(a, *v.shape, rows)
    with np.errstate(divide="ignore", invalid="ignore"):
        if dtype == "bf16":
            z = 448 * v / ax
        else:  # two fp32 roundings come before the code's
            z = ((np.float32(448) * v.astype(np.float32)) / ax.astype(np.float32)).astype(np.float64)
    return _e4m3(np.where(ax > 0, z, 0)), (a.astype(np.float32) / np.float32(448)).astype(np.float64)


def _rows(seed, M, C):
    x = synth.normal(seed, 1, M * C).reshape(M, C) * np.exp(synth.normal(seed, 2, C))
    return x * np.exp(0.5 * synth.normal(seed, 3, M))[:, None]


# ---------------------------------------------------------------------------
# residual add + RMSNorm

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [16, 48, 128, 208, 256, 1040, 1280, 2048, 2320, 4096])
@pytest.mark.parametrize("M,res", [(1, True), (77, True), (30, False)])
def test_add_rmsnorm(nc, dtype, C, M, res):
    import torch
    code = nc.NC_BF16 if dtype == "bf16" else nc.NC_F32
    xd, xv = _dev(_rows(C + M, M, C), dtype)
    rd, rv = _dev(synth.normal(C, 4, M * C).reshape(M, C) * 0.3, dtype)
    want = _dev(xv + rv, dtype)[1] if res else xv   # bf16 and fp32 sums of two values are exact in fp64: one rounding
    xo = torch.full_like(xd, 7)
    q = torch.zeros(M, C, dtype=torch.float8_e4m3fn, device="cuda")
    lds = M + 3
    s = torch.full((_blocks(C), lds), -1.0, device="cuda")
    r = torch.empty(M, device="cuda")
    assert nc.nc_add_rmsnorm_fp8(xd.data_ptr(), rd.data_ptr() if res else None, xo.data_ptr(), q.data_ptr(),
                                 s.data_ptr(), lds, r.data_ptr(), M, C, code, _stream()) == 0
    np.testing.assert_array_equal(_host(xo), want)
    np.testing.assert_array_equal(_host(q), _codes(want, 1, dtype)[0])
    r_ref = 1 / np.sqrt((want * want).mean(1) + EPS)
    adds = 8 * -(-C // 256) + 5
    tol_r = ((adds + 1) / 2 + 1 + 4) * U
    np.testing.assert_allclose(_host(r), r_ref, rtol=tol_r)
    s_ref = _block_max(want, 1) * r_ref / 448
    np.testing.assert_allclose(_host(s)[:, :M], s_ref, rtol=tol_r + 3 * U)
    assert (s[:, M:] == -1).all()  # nothing between the rows of scales
    # in place, on either operand, without r: the same bits
    for where in ("x", "res") if res else ("x",):
        xi, ri = xd.clone(), rd.clone()
        out = xi if where == "x" else ri
        q2, s2 = torch.zeros_like(q), torch.full_like(s, -1.0)
        assert nc.nc_add_rmsnorm_fp8(xi.data_ptr(), ri.data_ptr() if res else None, out.data_ptr(), q2.data_ptr(),
                                     s2.data_ptr(), lds, None, M, C, code, _stream()) == 0
        assert torch.equal(out, xo) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


def test_add_rmsnorm_special_rows(nc):
    import torch
    M, C = 6, 384
    x = np.ones((M, C))
    x[0] = 0                      # a row of zeros
    x[1, 128:256] = 0             # a block of zeros
    x[2, 130] = np.nan
    x[3, 5] = np.inf
    x[4] = 1e-30                  # far below eps
    xd, xv = _dev(x, "bf16")
    q = torch.zeros(M, C, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(3, M, device="cuda")
    r = torch.empty(M, device="cuda")
    assert nc.nc_add_rmsnorm_fp8(xd.data_ptr(), None, xd.data_ptr(), q.data_ptr(), s.data_ptr(), M, r.data_ptr(), M, C,
                                 nc.NC_BF16, _stream()) == 0
    qv, sv = _host(q), _host(s)
    y = qv * _expand(sv, M, C, 1)
    assert (qv[0] == 0).all() and (sv[:, 0] == 0).all()
    assert (y[1, 128:256] == 0).all() and sv[1, 1] == 0
    assert np.isnan(y[2]).all()
    assert np.isnan(y[3, :128]).all()
    np.testing.assert_allclose(y[4], xv[4] / np.sqrt(xv[4] ** 2 + EPS), rtol=1e-5)
    np.testing.assert_allclose(y[5], 1 / np.sqrt(1 + EPS), rtol=1e-5)


# ---------------------------------------------------------------------------
# quantiser

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 16), (1, 1280), (127, 144), (128, 128), (129, 272), (300, 2048), (33, 6160)])
def test_quant(nc, dtype, rows, R, K):
    import torch
    xd, xv = _dev(_rows(R + K, R, K + 16), dtype)  # a row stride beyond the columns
    xv = xv[:, :K]
    q = torch.full((R, K + 32), 3.0, device="cuda").to(torch.float8_e4m3fn)
    shape = (_blocks(K), R + 5) if rows == 1 else (-(-R // 128), _blocks(K) + 2)
    s = torch.full(shape, -1.0, device="cuda")
    assert nc.nc_quant_fp8(xd.data_ptr(), K + 16, q.data_ptr(), K + 32, s.data_ptr(), shape[1], R, K, rows,
                           nc.NC_BF16 if dtype == "bf16" else nc.NC_F32, _stream()) == 0
    cq, cs = _codes(xv, rows, dtype)
    np.testing.assert_array_equal(_host(q)[:, :K], cq)
    assert (_host(q)[:, K:] == 3).all()
    np.testing.assert_array_equal(_host(s)[:, :cs.shape[1]], cs)
    assert (s[:, cs.shape[1]:] == -1).all()


def test_quant_every_bf16_quotient(nc):
    # every pair of 8-bit significands, over every exponent that reaches a code: all ties and borders
    sig = (128 + np.arange(128)) / 128.0
    exps = np.arange(0, -20, -1)
    x = np.zeros((128, len(exps) * 2 * 128))
    for j, e in enumerate(exps):
        for h in range(2):
            b = x[:, (2 * j + h) * 128:(2 * j + h + 1) * 128]
            b[:, 0] = sig                                      # the block's largest
            v = np.where(sig[None] * 2.0 ** e <= sig[:, None], sig[None] * 2.0 ** e, 0)  # nothing above it
            b[:, 1:] = (v[:, 1:] if h == 0 else -v[:, :-1])
    import torch
    R, K = x.shape
    xd, xv = _dev(x, "bf16")
    np.testing.assert_array_equal(xv, x)
    q = torch.zeros(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(_blocks(K), R, device="cuda")
    assert nc.nc_quant_fp8(xd.data_ptr(), K, q.data_ptr(), K, s.data_ptr(), R, R, K, 1, nc.NC_BF16, _stream()) == 0
    cq, cs = _codes(x, 1)
    np.testing.assert_array_equal(_host(q), cq)
    np.testing.assert_array_equal(_host(s), cs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant_extremes(nc, dtype, rows):
    import torch
    R, K = 128, 1024
    x = np.zeros((R, K))
    pat = np.linspace(-1, 1, 128)
    for j, scale in enumerate([1e-36, 2.0 ** -110, 1.0, 1e30, 3e38]):
        x[:, 128 * j:128 * j + 128] = pat * scale
    x[:, 640:768] = 0
    x[0, 768] = np.nan
    x[1:, 768:896] = 1.0
    x[0, 900] = np.inf
    xd, xv = _dev(x, dtype)
    q = torch.zeros(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((8, R) if rows == 1 else (1, 8), device="cuda")
    assert nc.nc_quant_fp8(xd.data_ptr(), K, q.data_ptr(), K, s.data_ptr(), s.shape[1], R, K, rows,
                           nc.NC_BF16 if dtype == "bf16" else nc.NC_F32, _stream()) == 0
    a = _block_max(xv[:, :768], rows)
    ax = _expand(a, R, 768, rows)
    qv = _host(q)
    # the scaling up and down by a power of two is exact: the quotient's one or two roundings are as in the normal range
    z = np.where(ax > 0, 448 * (xv[:, :768] / np.where(ax > 0, ax, 1)), 0)
    near = np.abs(qv[:, :768] - z) <= np.maximum(np.abs(z) * 2.0 ** -4, 2.0 ** -10) * (1 + 4 * U)
    assert near.all()
    np.testing.assert_array_equal(np.abs(qv[:, :640]).max(1), 448)
    assert (qv[:, 640:768] == 0).all()
    with np.errstate(invalid="ignore"):
        y = qv * _expand(_host(s), R, K, rows)
    assert np.isnan(y[0, 768]) and np.isnan(y[0, 900])
    # the code of 1 is 448 and its scale RN(1 / 448): their product is 1 within the scale's half step
    assert (np.abs(y[1:, 768:896] - 1) <= U).all()


# ---------------------------------------------------------------------------
# product

def _operand(seed, R, K, rows, ld):
    """e4m3 codes [R, ld] with scales, and the values they stand for."""
    import torch
    v = _rows(seed, R, K) if rows == 1 else synth.normal(seed, 5, R * K).reshape(R, K) / np.sqrt(K)
    c, s = _codes(_dev(v, "bf16")[1], rows)
    buf = np.full((R, ld), 2.0, dtype=np.float32)  # what lies between the rows must not count
    buf[:, :K] = c
    q = torch.from_numpy(buf).cuda().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(_host(q)[:, :K], c)
    return q, s, c * _expand(s, R, K, rows)


def _acc_bound(av, bv):
    kb = _blocks(av.shape[1])
    mag = np.abs(av) @ np.abs(bv).T
    return mag, (128 * 2 + 4 * kb) * U * mag


def _case(nc, M, N, K, seed=0, pad=16):
    import torch
    up16 = lambda n: -(-n // 16) * 16  # noqa: E731
    lda, ldb = up16(K) + pad, up16(K) + 2 * pad
    a, sa, av = _operand(seed + M, M, K, 1, lda)
    b, sb, bv = _operand(seed + 7 * N, N, K, 128, ldb)
    lsa, lsb = M + 5, _blocks(K) + 1
    sad = torch.full((_blocks(K), lsa), float("nan"), device="cuda")
    sad[:, :M] = torch.from_numpy(sa.copy()).float()
    sbd = torch.full((_blocks(N), lsb), float("nan"), device="cuda")
    sbd[:, :_blocks(K)] = torch.from_numpy(sb.copy()).float()
    return dict(a=a, lda=lda, sa=sad, lsa=lsa, b=b, ldb=ldb, sb=sbd, lsb=lsb, av=av, bv=bv, M=M, N=N, K=K)


def _gemm(nc, c, epi, D, ldd, sd=None, lsd=0, stream=None):
    return nc.nc_gemm_fp8(c["a"].data_ptr(), c["lda"], c["sa"].data_ptr(), c["lsa"], c["b"].data_ptr(), c["ldb"],
                          c["sb"].data_ptr(), c["lsb"], D.data_ptr(), ldd, sd.data_ptr() if sd is not None else None,
                          lsd, c["M"], c["N"], c["K"], getattr(nc, "NC_EPI_" + epi),
                          _stream() if stream is None else stream)


def _check(nc, c, epi, refs=None):
    import torch
    M, N = c["M"], c["N"]
    acc, (mag, e) = refs if refs else (c["av"] @ c["bv"].T, _acc_bound(c["av"], c["bv"]))
    ldd = -(-N // 16) * 16 + 16
    if epi == "STORE_F32":
        D = torch.full((M + 1, ldd), 7.0, device="cuda")
    elif epi == "RELU2_FP8":
        D = torch.full((M + 1, ldd), 7.0, device="cuda").to(torch.float8_e4m3fn)
    else:
        D = _dev(synth.normal(3, 3, (M + 1) * ldd).reshape(M + 1, ldd) * 2, "bf16")[0]
    D0 = _host(D)
    lsd = M + 3
    sd = torch.full((_blocks(N), lsd), -1.0, device="cuda")
    assert _gemm(nc, c, epi, D, ldd, sd, lsd) == 0
    assert nc.nc_ops_status(_stream(), 60000) == 0
    got = _host(D)
    np.testing.assert_array_equal(got[:, N:], D0[:, N:])   # nothing past N
    np.testing.assert_array_equal(got[M:], D0[M:])         # nothing past M
    got = got[:M, :N]
    relu2 = np.maximum(acc, 0) ** 2
    e2 = 2 * np.abs(acc) * e + e * e + U * relu2
    if epi == "RELU2_FP8":
        s = _host(sd)[:, :M]
        assert (sd[:, M:] == -1).all()
        amax, emax = _block_max(relu2, 1), _block_max(e2, 1)
        assert (np.abs(s - amax / 448) <= emax / 448 + 2 * U * amax / 448).all()
        sx = _expand(s, M, N, 1)
        # the code is the nearest to 448 v / a, v and a each within their bounds (v <= a)
        tol = e2 + _expand(emax, M, N, 1) + np.maximum(2.0 ** -4 * (relu2 + e2), 2.0 ** -10 * sx) * (1 + 8 * U)
        assert (np.abs(got * sx - relu2) <= tol).all()
        return D, sd
    assert (sd == -1).all()
    if epi == "STORE_F32":
        ref, tol = acc, e
    elif epi == "RELU2":
        ref, tol = relu2, e2
    elif epi == "SOFTCAP":
        ref, tol = 15 * np.tanh(acc / 15), e + 15 * 2.0 ** -19
    elif epi == "ADD":
        ref = D0[:M, :N] + acc
        tol = e + U * np.abs(ref)
    else:
        ref, tol = acc, e
    if epi != "STORE_F32":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    worst = np.max(np.abs(got - ref) - tol)
    assert (np.abs(got - ref) <= tol).all(), worst
    return D, sd


EPIS = ["STORE", "STORE_F32", "ADD", "RELU2", "SOFTCAP", "RELU2_FP8"]

SHAPES = [
    # M, N, K
    (1, 1, 1), (1, 16, 128), (1, 1536, 1280), (2, 130, 272), (16, 1000, 640), (17, 257, 1040), (32, 128, 144),
    (33, 300, 2048), (64, 129, 384), (65, 513, 512), (127, 128, 4096), (128, 640, 1280), (129, 64, 48),
    (200, 1003, 656), (300, 520, 1040), (515, 776, 1296), (1030, 264, 272), (270, 200, 8208),
    (20485, 392, 272),     # several tiles per pair of CTAs, the last column half of 8 columns
    (300, 1003, 272), (290, 5, 144), (513, 385, 130), (300, 262, 16),   # N that no 16-byte unit divides
    (1000, 500, 1100), (4000, 128, 1040), (300, 1280, 1296), (260, 4608, 1040),   # 128-row tiles with K cut, and not
    (100, 10241, 400), (256, 9600, 272),   # 256-row tiles for fewer rows
    (270, 300, 3200), (400, 1003, 6416),   # K cut over two and four pairs of CTAs
    (40, 20485, 144),      # many weight tiles
    (16, 40003, 272), (5, 38400, 1040),   # more tiles than two CTAs per SM hold
]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(nc, M, N, K):
    c = _case(nc, M, N, K)
    refs = (c["av"] @ c["bv"].T, _acc_bound(c["av"], c["bv"]))
    for epi in EPIS:
        _check(nc, c, epi, refs)


def _random_case(i):
    """Sizes over the whole range, small ones as often as large (no size is special to a kernel)."""
    r = np.random.RandomState(1000 + i)
    M = int(np.exp(r.uniform(0, np.log(1500))))
    N = int(np.exp(r.uniform(0, np.log(4000))))
    K = int(np.exp(r.uniform(0, np.log(5000))))
    return M, N, K, EPIS[i % len(EPIS)]


@pytest.mark.parametrize("i", range(48))
def test_gemm_random_sizes(nc, i):
    M, N, K, epi = _random_case(i)
    c = _case(nc, M, N, K, seed=i, pad=16 * (i % 3))
    _check(nc, c, epi)


@pytest.mark.parametrize("M,N", [(1, 40), (70, 300), (300, 520)])
def test_gemm_zero_blocks(nc, M, N):
    """Rows and weight blocks of zeros (scale 0) give zeros, in 8 bits too."""
    import torch
    c = _case(nc, M, N, 400)
    c["a"].view(torch.uint8)[0] = 0
    c["sa"][:, 0] = 0
    D = torch.full((M, 16 * -(-N // 16)), 3.0, device="cuda").bfloat16()
    assert _gemm(nc, c, "STORE", D, D.shape[1]) == 0
    assert (D[0, :N] == 0).all() and (D[1:, :N] != 0).any() == (M > 1)
    q = torch.full((M, 16 * -(-N // 16)), 3.0, device="cuda").to(torch.float8_e4m3fn)
    sd = torch.full((_blocks(N), M), 5.0, device="cuda")
    assert _gemm(nc, c, "RELU2_FP8", q, q.shape[1], sd, M) == 0
    assert (q.float()[0, :N] == 0).all() and (sd[:, 0] == 0).all()
    # a product that is negative everywhere: relu^2 leaves zeros
    c["a"].view(torch.uint8).fill_(0x38)      # 1
    c["b"].view(torch.uint8).fill_(0xb8)      # -1
    c["sa"].fill_(0.5)
    c["sb"].fill_(0.25)
    assert _gemm(nc, c, "RELU2_FP8", q, q.shape[1], sd, M) == 0
    assert (q.float()[:, :N] == 0).all() and (sd == 0).all()
    assert _gemm(nc, c, "STORE", D, D.shape[1]) == 0
    assert (D[:, :N] == -50).all()            # 400 products of -1/8, exact


@pytest.mark.parametrize("M,N", [(9, 200), (300, 300)])
def test_gemm_tiny_and_huge_scales(nc, M, N):
    """Sums far from 1: an 8-bit output of sums near 2^-70 (their squares near 2^-140, below any normal
    number's square root) and of sums near 2^50."""
    import torch
    K = 256
    c = _case(nc, M, N, K)
    sa0 = c["sa"].clone()
    for e in (-50, 50):
        c["sa"].copy_(sa0 * 2.0 ** e)
        D = torch.zeros(M, 16 * -(-N // 16), device="cuda").to(torch.float8_e4m3fn)
        sd = torch.zeros(_blocks(N), M, device="cuda")
        assert _gemm(nc, c, "RELU2_FP8", D, D.shape[1], sd, M) == 0
        acc = (c["av"] * 2.0 ** e) @ c["bv"].T
        v = np.maximum(acc, 0) ** 2
        _, ea = _acc_bound(c["av"] * 2.0 ** e, c["bv"])
        ev = 2 * np.abs(acc) * ea + ea * ea + U * v
        s = _host(sd)
        sx = _expand(s, M, N, 1)
        # scales below 2^-126 have steps of 2^-149
        tol = ev + _expand(_block_max(ev, 1), M, N, 1) + np.maximum(2.0 ** -4 * (v + ev), 2.0 ** -10 * sx) * (1 + 8 * U)
        assert (np.abs(_host(D)[:, :N] * sx - v) <= tol + 448 * 2.0 ** -149).all()


def test_offsets_past_32_bits(nc):
    """Rows that start past 2^31 and 2^32 elements, in every operator."""
    import torch
    bf, e8 = torch.bfloat16, torch.float8_e4m3fn
    M, C, tail = 2_200_000, 2048, 5
    x = torch.zeros(M, C, dtype=bf, device="cuda")
    xt, xv = _dev(_rows(11, tail, C), "bf16")
    x[-tail:] = xt
    cq, cs = _codes(xv, 1)
    q = torch.zeros(M, C, dtype=e8, device="cuda")
    s = torch.zeros(_blocks(C), M, device="cuda")
    assert nc.nc_quant_fp8(x.data_ptr(), C, q.data_ptr(), C, s.data_ptr(), M, M, C, 1, nc.NC_BF16, _stream()) == 0
    np.testing.assert_array_equal(_host(q[-tail:]), cq)
    np.testing.assert_array_equal(_host(s[:, -tail:]), cs)
    s128 = torch.zeros(-(-M // 128), _blocks(C), device="cuda")
    q.zero_()
    assert nc.nc_quant_fp8(x.data_ptr(), C, q.data_ptr(), C, s128.data_ptr(), _blocks(C), M, C, 128, nc.NC_BF16,
                           _stream()) == 0
    last = M - M % 128
    assert M - last >= tail
    block = np.zeros((M - last, C))
    block[-tail:] = xv
    bq, bs = _codes(block, 128)
    np.testing.assert_array_equal(_host(q[last:]), bq)
    np.testing.assert_array_equal(_host(s128[-1:]), bs)
    assert nc.nc_add_rmsnorm_fp8(x.data_ptr(), x.data_ptr(), x.data_ptr(), q.data_ptr(), s.data_ptr(), M, None, M, C,
                                 nc.NC_BF16, _stream()) == 0
    np.testing.assert_array_equal(_host(x[-tail:]), 2 * xv)
    np.testing.assert_array_equal(_host(q[-tail:]), cq)
    del x, s128
    # D past 2^32 elements: A = the last rows' codes in one K block, weights of one block
    K, N = 128, 2000
    w, sw, wv = _operand(5, N, K, 128, K)
    swd = torch.from_numpy(sw.copy()).float().cuda()
    a = q[:, :K]
    D = torch.empty(M, N, dtype=bf, device="cuda")
    s1 = s[:1].contiguous()
    assert nc.nc_gemm_fp8(a.data_ptr(), C, s1.data_ptr(), M, w.data_ptr(), K, swd.data_ptr(), 1, D.data_ptr(), N, None, 0,
                          M, N, K, nc.NC_EPI_STORE, _stream()) == 0
    assert nc.nc_ops_status(_stream(), 60000) == 0
    av = _host(a[-tail:]) * _host(s1[:, -tail:]).T
    ref, (_, e) = av @ wv.T, _acc_bound(av, wv)
    got = _host(D[-tail:])
    assert (np.abs(got - ref) <= e + 2.0 ** -8 * (np.abs(ref) + e)).all()
    assert (D[:-tail:99991] == 0).all()


def test_calls_on_two_streams_at_once(nc):
    """Both kinds of kernel on two streams at once, again and again: each call's bits are those of the call alone."""
    import torch
    shapes = [(900, 1300, 1040, "STORE"), (5, 2000, 2048, "RELU2"), (40, 700, 1300, "STORE_F32"), (300, 600, 6416, "SOFTCAP"),
              (150, 256, 2048, "STORE")]
    cases = [(_case(nc, M, N, K), epi) for M, N, K, epi in shapes]

    def out(c, epi):
        return torch.zeros(c["M"], 16 * -(-c["N"] // 16), device="cuda",
                           dtype=torch.float32 if epi == "STORE_F32" else torch.bfloat16)
    want = []
    for c, epi in cases:
        D = out(c, epi)
        assert _gemm(nc, c, epi, D, D.shape[1]) == 0
        want.append(D)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[[out(c, epi) for c, epi in cases] for _ in range(4)] for _ in streams]
    torch.cuda.synchronize()
    for r in range(4):
        for i in range(len(cases)):
            for k, st in enumerate(streams):
                j = (i + 2 * k) % len(cases)
                c, epi = cases[j]
                assert _gemm(nc, c, epi, got[k][r][j], got[k][r][j].shape[1], stream=st.cuda_stream) == 0
    torch.cuda.synchronize()
    for k in range(2):
        for r in range(4):
            for j, w in enumerate(want):
                assert torch.equal(got[k][r][j], w), (k, r, j)
    assert nc.nc_ops_status(_stream(), 60000) == 0


def test_gemm_repeats_bit_for_bit(nc):
    import torch
    for M, N, K in [(3, 1536, 1280), (300, 520, 1040), (700, 1300, 2048)]:
        c = _case(nc, M, N, K)
        for epi in EPIS:
            (d1, s1), (d2, s2) = _check(nc, c, epi), _check(nc, c, epi)
            assert torch.equal(d1.view(torch.uint8), d2.view(torch.uint8)) and torch.equal(s1, s2)


@pytest.mark.parametrize("M,N", [(20, 300), (600, 520)])
def test_gemm_nan_stays_in_its_row_and_column(nc, M, N):
    import torch
    K = 400
    c = _case(nc, M, N, K)
    c["a"].view(torch.uint8)[3, 130] = 0x7f        # a NaN code in row 3
    c["sa"][1, 5] = float("nan")                   # a NaN scale of row 5
    c["b"].view(torch.uint8)[7, 399] = 0xff        # a NaN code in weight row 7
    for epi in EPIS[:5]:
        D = torch.zeros(M, 16 * -(-N // 16), device="cuda", dtype=torch.float32 if epi == "STORE_F32" else torch.bfloat16)
        assert _gemm(nc, c, epi, D, D.shape[1]) == 0
        bad = torch.isnan(D[:, :N]).cpu().numpy()
        want = np.zeros((M, N), bool)
        want[[3, 5]] = True
        want[:, 7] = True
        np.testing.assert_array_equal(bad, want, err_msg=epi)
    D = torch.zeros(M, 16 * -(-N // 16), device="cuda").to(torch.float8_e4m3fn)
    sd = torch.zeros(_blocks(N), M, device="cuda")
    assert _gemm(nc, c, "RELU2_FP8", D, D.shape[1], sd, M) == 0
    bad = np.isnan(_host(D)[:, :N] * _expand(_host(sd), M, N, 1))
    np.testing.assert_array_equal(bad, want)


# ---------------------------------------------------------------------------
# together

def _mlp_inputs(M, C, F):
    x, xv = _dev(_rows(M, M, C), "bf16")
    res, rv = _dev(0.3 * synth.normal(M, 9, M * C).reshape(M, C), "bf16")
    w1, w1v = _dev(synth.normal(1, 6, F * C).reshape(F, C) / np.sqrt(C), "bf16")
    w2, w2v = _dev(synth.normal(2, 6, F * C).reshape(C, F) / np.sqrt(F), "bf16")
    return (x, res, w1, w2), (xv, rv, w1v, w2v)


def _mlp_buffers(M, C, F):
    import torch
    e8 = torch.float8_e4m3fn
    def f(*n):
        return torch.full(n, float("nan"), device="cuda")
    return dict(xo=f(M, C).bfloat16(), q=f(M, C).to(e8), s=f(_blocks(C), M), h=f(M, F).to(e8), sh=f(_blocks(F), M),
                w1=f(F, C).to(e8), s1=f(_blocks(F), _blocks(C)), w2=f(C, F).to(e8), s2=f(_blocks(C), _blocks(F)))


def _mlp_weights(nc, t, b, C, F, st):
    assert nc.nc_quant_fp8(t[2].data_ptr(), C, b["w1"].data_ptr(), C, b["s1"].data_ptr(), _blocks(C), F, C, 128,
                           nc.NC_BF16, st) == 0
    assert nc.nc_quant_fp8(t[3].data_ptr(), F, b["w2"].data_ptr(), F, b["s2"].data_ptr(), _blocks(F), C, F, 128,
                           nc.NC_BF16, st) == 0


def _mlp(nc, t, b, M, C, F, st):
    assert nc.nc_add_rmsnorm_fp8(t[0].data_ptr(), t[1].data_ptr(), b["xo"].data_ptr(), b["q"].data_ptr(),
                                 b["s"].data_ptr(), M, None, M, C, nc.NC_BF16, st) == 0
    assert nc.nc_gemm_fp8(b["q"].data_ptr(), C, b["s"].data_ptr(), M, b["w1"].data_ptr(), C, b["s1"].data_ptr(),
                          _blocks(C), b["h"].data_ptr(), F, b["sh"].data_ptr(), M, M, F, C, nc.NC_EPI_RELU2_FP8, st) == 0
    assert nc.nc_gemm_fp8(b["h"].data_ptr(), F, b["sh"].data_ptr(), M, b["w2"].data_ptr(), F, b["s2"].data_ptr(),
                          _blocks(F), b["xo"].data_ptr(), C, None, 0, M, C, F, nc.NC_EPI_ADD, st) == 0


@pytest.mark.parametrize("M", [1, 40, 333, 1100])
def test_mlp_of_a_block(nc, M):
    """norm, up-projection and down-projection as a block runs them: every stage
    against the 64-bit definition on the stage's own operands, and the whole
    against the unquantised block within the codes' steps."""
    C, F = 256, 1024
    t, (xv, rv, w1v, w2v) = _mlp_inputs(M, C, F)
    b = _mlp_buffers(M, C, F)
    _mlp_weights(nc, t, b, C, F, _stream())
    _mlp(nc, t, b, M, C, F, _stream())
    assert nc.nc_ops_status(_stream(), 60000) == 0
    x1 = _dev(xv + rv, "bf16")[1]
    y, _ = oracle.rmsnorm(x1)
    q = _host(b["q"]) * _expand(_host(b["s"]), M, C, 1)
    w1 = _host(b["w1"]) * _expand(_host(b["s1"]), F, C, 128)
    w2 = _host(b["w2"]) * _expand(_host(b["s2"]), C, F, 128)
    h = _host(b["h"]) * _expand(_host(b["sh"]), M, F, 1)

    def code_error(v, rows):  # half a step of each code, and the fp32 roundings of its scale
        return np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * _expand(_block_max(v, rows), *v.shape, rows) / 448) + 1e-5 * np.abs(v)
    assert (np.abs(q - y) <= code_error(y, 1)).all()
    assert (np.abs(w1 - w1v) <= code_error(w1v, 128)).all() and (np.abs(w2 - w2v) <= code_error(w2v, 128)).all()
    # on the stages' own operands
    acc, (_, e) = q @ w1.T, _acc_bound(q, w1)
    v = np.maximum(acc, 0) ** 2
    ev = 2 * np.abs(acc) * e + e * e + U * v
    sx = _expand(_host(b["sh"]), M, F, 1)
    tol = ev + _expand(_block_max(ev, 1), M, F, 1) + np.maximum(2.0 ** -4 * (v + ev), 2.0 ** -10 * sx) * (1 + 8 * U)
    assert (np.abs(h - v) <= tol).all()
    ref, (_, e) = x1 + h @ w2.T, _acc_bound(h, w2)
    assert (np.abs(_host(b["xo"]) - ref) <= e + (2.0 ** -8 + U) * (np.abs(ref) + e)).all()
    # against the unquantised MLP: the errors of the operands through the products
    ey, e1, e2 = code_error(y, 1), code_error(w1v, 128), code_error(w2v, 128)
    a_ref = y @ w1v.T
    ea = ey @ np.abs(w1v).T + np.abs(y) @ e1.T + ey @ e1.T + e.max() * 0
    v_ref = np.maximum(a_ref, 0) ** 2
    ev = 2 * np.abs(a_ref) * ea + ea * ea
    eh = ev + 2.0 ** -4 * (v_ref + ev) + 2.0 ** -10 * _expand(_block_max(v_ref + ev, 1), M, F, 1) / 448
    ex = eh @ np.abs(w2v).T + v_ref @ e2.T + eh @ e2.T
    ref = x1 + v_ref @ w2v.T
    assert (np.abs(_host(b["xo"]) - ref) <= 1.01 * ex + 2.0 ** -8 * (np.abs(ref) + ex)).all()


@pytest.mark.parametrize("M", [3, 150, 700])
def test_chain_of_calls_without_waiting(nc, M):
    """Forty MLPs in a row on the same stream buffers, each call's operands the last one's results: the bits are
    those of the same calls waited for one by one (a call that reads before the one ahead of it has written, or
    writes what that one still reads, shows), eager and replayed from a graph."""
    import torch
    C, F, n = 256, 1024, 40
    t, _ = _mlp_inputs(M, C, F)
    b = _mlp_buffers(M, C, F)
    _mlp_weights(nc, t, b, C, F, _stream())
    x0 = t[0].clone()

    def step(wait):
        # x += xo and its norm's codes feed the products (unnormalised, relu^2 would square x at every step: no finite
        # chain); the quantiser before writes the same codes' place, for the norm to write over
        st = _stream()
        calls = [
            lambda: nc.nc_quant_fp8(t[0].data_ptr(), C, b["q"].data_ptr(), C, b["s"].data_ptr(), M, M, C, 1, nc.NC_BF16, st),
            lambda: nc.nc_add_rmsnorm_fp8(t[0].data_ptr(), b["xo"].data_ptr(), t[0].data_ptr(), b["q"].data_ptr(),
                                          b["s"].data_ptr(), M, None, M, C, nc.NC_BF16, st),
            lambda: nc.nc_gemm_fp8(b["q"].data_ptr(), C, b["s"].data_ptr(), M, b["w1"].data_ptr(), C, b["s1"].data_ptr(),
                                   _blocks(C), b["h"].data_ptr(), F, b["sh"].data_ptr(), M, M, F, C, nc.NC_EPI_RELU2_FP8, st),
            lambda: nc.nc_gemm_fp8(b["h"].data_ptr(), F, b["sh"].data_ptr(), M, b["w2"].data_ptr(), F, b["s2"].data_ptr(),
                                   _blocks(F), b["xo"].data_ptr(), C, None, 0, M, C, F, nc.NC_EPI_STORE, st)]
        for c in calls:
            assert c() == 0
            if wait:
                torch.cuda.synchronize()
        t[0].mul_(0.5)  # another kind of kernel between
        if wait:
            torch.cuda.synchronize()

    def run(wait):
        t[0].copy_(x0)
        b["xo"].zero_()
        for _ in range(n):
            step(wait)
        torch.cuda.synchronize()
        return t[0].clone(), b["q"].view(torch.uint8).clone(), b["h"].view(torch.uint8).clone()
    want = run(True)
    assert torch.isfinite(want[0].float()).all() and (want[0] != 0).any()
    for _ in range(3):
        for w, g in zip(want, run(False)):
            assert torch.equal(w, g)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(n):
            step(False)
    t[0].copy_(x0)
    b["xo"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(t[0], want[0]) and torch.equal(b["h"].view(torch.uint8), want[2])
    assert nc.nc_ops_status(_stream(), 60000) == 0


def test_mlp_on_streams_and_in_graphs(nc):
    """The same run on a side stream, and captured twice into graphs whose replays overlap on two streams with
    buffers of their own: bit for bit the eager result on the default stream."""
    import torch
    M, C, F = 300, 256, 1024
    t, _ = _mlp_inputs(M, C, F)
    b0 = _mlp_buffers(M, C, F)
    _mlp_weights(nc, t, b0, C, F, _stream())
    _mlp(nc, t, b0, M, C, F, _stream())
    torch.cuda.synchronize()
    want = b0["xo"].clone()
    side = torch.cuda.Stream()
    b1 = _mlp_buffers(M, C, F)
    torch.cuda.synchronize()
    _mlp_weights(nc, t, b1, C, F, side.cuda_stream)
    _mlp(nc, t, b1, M, C, F, side.cuda_stream)
    side.synchronize()
    assert torch.equal(b1["xo"], want)
    graphs, bufs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        b = _mlp_buffers(M, C, F)
        _mlp_weights(nc, t, b, C, F, _stream())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _mlp(nc, t, b, M, C, F, _stream())
        graphs.append(g)
        bufs.append(b)
    for _ in range(5):
        for b in bufs:
            b["xo"].zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for b in bufs:
            assert torch.equal(b["xo"], want)
    assert nc.nc_ops_status(_stream(), 60000) == 0
