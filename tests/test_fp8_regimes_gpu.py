"""nc_gemm_fp8 in every form that its sizes choose: kernel, rows a tile, CTAs
that share K, tiles a pair of CTAs takes.  A CPU test holds REGIMES against the
rule, so that none can drop out of these tests unseen."""
import numpy as np
import pytest

import test_fp8_gpu as base

nc = base.nc

# (pair, rows of activations a tile, four CTAs per SM, splits of K): sizes
REGIMES = {
    (False, 16, True, 1): [(7, 38100, 300)],
    (False, 16, False, 1): [(3, 300, 23), (13, 20010, 400)],
    (False, 16, False, 2): [(5, 300, 350)],
    (False, 16, False, 4): [(11, 301, 514)],
    (False, 16, False, 8): [(2, 1314, 1010)],
    (False, 32, False, 1): [(17, 318, 20), (29, 20010, 400)],
    (False, 32, False, 2): [(21, 338, 339)],
    (False, 32, False, 4): [(31, 335, 401)],
    (False, 32, False, 8): [(18, 1340, 1933)],
    (False, 64, False, 1): [(33, 308, 51), (61, 20010, 400)],
    (False, 64, False, 2): [(40, 311, 376)],
    (False, 64, False, 4): [(63, 302, 445)],
    (False, 64, False, 8): [(36, 1327, 1913)],
    (False, 128, False, 1): [(65, 308, 40), (250, 301, 120)],
    (False, 128, False, 2): [(68, 314, 379)],
    (False, 128, False, 4): [(130, 1301, 482), (1299, 330, 1100)],
    (False, 128, False, 8): [(70, 1300, 1380), (301, 395, 1801)],
    (True, 0, False, 1): [(258, 314, 45), (4400, 4616, 912), (19300, 301, 1300)],   # one tile a pair; several, with
                                                                                   # whole and ragged groups of tiles and scales
    (True, 0, False, 2): [(513, 1100, 3200), (1000, 1003, 5000)],
    (True, 0, False, 4): [(400, 1300, 6416), (270, 1500, 7000)],
}
ALL = [(r, s) for r, sizes in REGIMES.items() for s in sizes]
CUT = [s for r, s in ALL if r[0] and r[3] > 1]


@pytest.mark.gpu
@pytest.mark.parametrize("regime,size", ALL)
def test_every_epilogue(nc, regime, size):
    c = base._case(nc, *size)
    refs = (c["av"] @ c["bv"].T, base._acc_bound(c["av"], c["bv"]))
    for epi in base.EPIS:
        base._check(nc, c, epi, refs)


@pytest.mark.gpu
@pytest.mark.parametrize("size", CUT)
def test_cut_pairs_repeat_bit_for_bit(nc, size):
    import torch
    c = base._case(nc, *size)
    refs = (c["av"] @ c["bv"].T, base._acc_bound(c["av"], c["bv"]))
    for epi in base.EPIS:
        d, s = base._check(nc, c, epi, refs)
        for _ in range(3):
            d2, s2 = base._check(nc, c, epi, refs)
            assert torch.equal(d.view(torch.uint8), d2.view(torch.uint8)) and torch.equal(s, s2)


def _out(c, epi):
    import torch
    return torch.zeros(c["M"], 16 * -(-c["N"] // 16), device="cuda",
                       dtype=torch.float32 if epi == "STORE_F32" else torch.bfloat16)


@pytest.mark.gpu
def test_regimes_on_two_streams_at_once(nc):
    """One size of every form with K cut, and uncut pairs, on two streams at once: each call's bits are those alone."""
    import torch
    sizes = [REGIMES[r][0] for r in REGIMES if r[3] > 1 and r[1] in (0, 16, 128)] + [(900, 1300, 1040)]
    epis = ["STORE", "RELU2", "STORE_F32", "SOFTCAP"]
    cases = [(base._case(nc, *s), epis[i % 4]) for i, s in enumerate(sizes)]
    want = []
    for c, epi in cases:
        D = _out(c, epi)
        assert base._gemm(nc, c, epi, D, D.shape[1]) == 0
        want.append(D)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[[_out(c, epi) for c, epi in cases] for _ in range(4)] for _ in streams]
    torch.cuda.synchronize()
    for r in range(4):
        for i in range(len(cases)):
            for k, st in enumerate(streams):
                j = (i + 3 * k) % len(cases)
                c, epi = cases[j]
                assert base._gemm(nc, c, epi, got[k][r][j], got[k][r][j].shape[1], stream=st.cuda_stream) == 0
    torch.cuda.synchronize()
    for k in range(2):
        for r in range(4):
            for j, w in enumerate(want):
                assert torch.equal(got[k][r][j], w), (k, r, sizes[j])
    assert nc.nc_ops_status(base._stream(), 60000) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,C,F", [(300, 1500, 6416), (700, 1008, 5008)])
def test_chain_of_cut_pairs(nc, M, C, F):
    """norm, up-projection and a down-projection whose K is cut over pairs, onto the stream itself, again and again without
    a wait and from a graph: the bits of the same calls waited for one by one."""
    import torch
    n, up = 12, lambda k: -(-k // 16) * 16  # noqa: E731
    e8, Cp, Fp = torch.float8_e4m3fn, up(C), up(F)
    g = torch.Generator(device="cuda").manual_seed(M)
    C, F = Cp, Fp
    x0 = torch.randn(M, C, device="cuda", generator=g).bfloat16()
    kb, fb = base._blocks(C), base._blocks(F)

    def weight(R, K):
        w = (torch.randn(R, K, device="cuda", generator=g) / K ** 0.5).bfloat16()
        q, s = torch.empty(R, K, device="cuda").to(e8), torch.empty(base._blocks(R), base._blocks(K), device="cuda")
        assert nc.nc_quant_fp8(w.data_ptr(), K, q.data_ptr(), K, s.data_ptr(), s.shape[1], R, K, 128, nc.NC_BF16,
                               base._stream()) == 0
        return q, s
    (w1, s1), (w2, s2) = weight(F, C), weight(C, F)
    torch.cuda.synchronize()
    x, q, h = x0.clone(), x0.to(e8), torch.zeros(M, F, device="cuda").to(e8)
    s, sh = torch.empty(kb, M, device="cuda"), torch.empty(fb, M, device="cuda")

    def step(wait):
        st = base._stream()
        for call in (
            lambda: nc.nc_add_rmsnorm_fp8(x.data_ptr(), None, x.data_ptr(), q.data_ptr(), s.data_ptr(), M, None, M, C,
                                          nc.NC_BF16, st),
            lambda: nc.nc_gemm_fp8(q.data_ptr(), C, s.data_ptr(), M, w1.data_ptr(), C, s1.data_ptr(), kb, h.data_ptr(), F,
                                   sh.data_ptr(), M, M, F, C, nc.NC_EPI_RELU2_FP8, st),
            lambda: nc.nc_gemm_fp8(h.data_ptr(), F, sh.data_ptr(), M, w2.data_ptr(), F, s2.data_ptr(), fb, x.data_ptr(), C,
                                   None, 0, M, C, F, nc.NC_EPI_ADD, st)):
            assert call() == 0
            if wait:
                torch.cuda.synchronize()

    def run(wait):
        x.copy_(x0)
        torch.cuda.synchronize()
        for _ in range(n):
            step(wait)
        torch.cuda.synchronize()
        return x.clone(), h.view(torch.uint8).clone()
    want = run(True)
    assert torch.isfinite(want[0].float()).all() and not torch.equal(want[0], x0)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, run(False)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            step(False)
    for _ in range(3):
        x.copy_(x0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(h.view(torch.uint8), want[1])
    assert nc.nc_ops_status(base._stream(), 60000) == 0
