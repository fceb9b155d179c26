"""csrc/fp8_plan.h, compiled by the host compiler: which kernel an 8-bit product takes, and the tile order."""
import collections
import ctypes
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decoder_only_transformer_nanochat_b200", "csrc")
SRC = r"""
#include "fp8_plan.h"
using namespace nc::tc8;
extern "C" {
void get_plan(int M, int N, int K, int sms, int64_t *out) {
  const Plan p = plan(M, N, K, sms);
  out[0] = p.pair; out[1] = p.tn; out[2] = p.many; out[3] = p.splits; out[4] = p.tiles;
  out[5] = p.pair ? 1 : rows_ctas(p.tn, p.many);
}
// how often each tile comes up
void count_tiles(int n_m, int n_n, int *seen) {
  const PairTiles t(n_m, n_n);
  for (int u = 0; u < n_m * n_n; ++u) {
    int m = -1, n = -1;
    t.tile(u, m, n);
    if (m >= 0 && m < n_m && n >= 0 && n < n_n) ++seen[m * n_n + n];
  }
}
uint32_t divided(uint32_t u, uint32_t d) { return ByHost(d).div(u); }
}
"""
Plan = collections.namedtuple("Plan", "pair tn many splits tiles per_sm")
_lib = None


def lib():
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
            open(src, "w").write(SRC)
            subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, src, "-o", so],
                           check=True)
            _lib = ctypes.CDLL(so)
        _lib.divided.restype = ctypes.c_uint32
        _lib.divided.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    return _lib


def plan(M, N, K, sms=148):
    out = (ctypes.c_int64 * 6)()
    lib().get_plan(M, N, K, sms, out)
    return Plan(bool(out[0]), out[1], bool(out[2]), *out[3:])
