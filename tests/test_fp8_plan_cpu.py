"""The choice of kernel of nc_gemm_fp8, its cut of K and its tile order (host arithmetic)."""
import ctypes

import numpy as np
import pytest

from _fp8_plan import lib, plan

# clusters that run at once on 148 SMs, by CTAs per SM and cluster size (cudaOccupancyMaxActiveClusters)
ROOM = {(1, 2): 74, (1, 4): 33, (1, 8): 15, (2, 2): 148, (2, 4): 71, (2, 8): 33}


def _cluster(p):
    return p.splits * (2 if p.pair else 1)


@pytest.mark.parametrize("M,N,K,splits", [
    (1536, 1536, 6144, 1),    # 36 tiles: as clusters of four they would take two turns
    (768, 1536, 6144, 2),     # 18: clusters of four, not of eight
    (1024, 1024, 6144, 2),    # 16
    (960, 960, 6144, 2),
    (768, 1280, 6144, 4),     # 15 clusters of eight
    (2816, 768, 4096, 2),     # 33 clusters of four
    (513, 1100, 3200, 2), (400, 1300, 6416, 4), (1024, 1280, 1280, 1),
])
def test_cut_of_pairs(M, N, K, splits):
    p = plan(M, N, K)
    assert p.pair and p.splits == splits, p


@pytest.mark.parametrize("M,N,K,tn,splits", [(128, 2048, 4096, 128, 4), (128, 1920, 4096, 128, 8), (256, 1024, 4096, 128, 4),
                                             (1, 1536, 1280, 16, 8), (1, 65536, 1280, 16, 1)])
def test_cut_of_rows(M, N, K, tn, splits):
    p = plan(M, N, K)
    assert not p.pair and (p.tn, p.splits) == (tn, splits), p


def test_cut_tiles_run_at_once():
    """Sizes over the whole range: wherever K is cut, all clusters find room at once, and each part has a K block."""
    r = np.random.RandomState(0)
    cut = 0
    for _ in range(40000):
        M = int(np.exp(r.uniform(0, np.log(40000))))
        N = int(np.exp(r.uniform(0, np.log(70000))))
        K = int(np.exp(r.uniform(0, np.log(17000))))
        p = plan(M, N, K)
        assert p.splits in (1, 2, 4, 8) and p.splits <= -(-K // 128)
        if p.pair:
            assert p.tiles == -(-M // 256) * -(-N // 256) and p.splits <= 4
        else:
            assert p.tiles == -(-N // 128) * -(-M // p.tn) and (p.tn == 128 or M <= p.tn)
        if p.splits > 1:
            cut += 1
            assert p.tiles <= ROOM[p.per_sm, _cluster(p)], (M, N, K, p)
    assert cut > 4000


def test_every_tile_comes_up_once():
    sizes = [1, 2, 3, 5, 15, 16, 17, 18, 19, 31, 32, 33, 50, 64, 100, 257]
    for n_m in sizes:
        for n_n in sizes:
            seen = (ctypes.c_int * (n_m * n_n))()
            lib().count_tiles(n_m, n_n, seen)
            assert all(s == 1 for s in seen), (n_m, n_n)


def test_division_by_reciprocal():
    r = np.random.RandomState(1)
    top = 2 ** 31 - 1
    for d in [1, 2, 3, 5, 7, 16, 17, 48, 272, 4096, 65537, 2 ** 20 - 1, 2 ** 26] + [int(x) for x in r.randint(1, 2 ** 26, 200)]:
        us = {0, 1, d - 1, d, d + 1, 2 * d - 1, top, top - 1, top // d * d, top // d * d - 1} | {int(x) for x in r.randint(0, top, 50)}
        for u in us:
            assert lib().divided(u, d) == u // d, (u, d)


def test_gpu_tests_reach_every_form():
    """What the rule can choose (over a wide sample of sizes) is what the GPU tests' sizes make it choose."""
    regimes = pytest.importorskip("test_fp8_regimes_gpu").REGIMES
    for regime, sizes in regimes.items():
        for s in sizes:
            assert tuple(plan(*s)[:4]) == regime, (s, plan(*s))
    r = np.random.RandomState(5)
    seen = set()
    for _ in range(40000):
        seen.add(tuple(plan(*(int(np.exp(r.uniform(0, np.log(t)))) for t in (40000, 70000, 17000)))[:4]))
    assert seen == set(regimes)
    # tiles of pairs whose K is not cut: several a pair of CTAs, in whole and partial groups of 16, over a ragged second
    # group of five K blocks
    assert any(plan(M, N, K).tiles > 2 * 74 and N > 16 * 256 and M > 16 * 256 and -(-M // 256) % 16 and -(-K // 128) % 5
               for M, N, K in regimes[(True, 0, False, 1)])
    for M, C, F in ((300, 1504, 6416), (700, 1008, 5008)):  # the chain's down-projections
        assert plan(M, C, F).pair and plan(M, C, F).splits > 1
