"""csrc/kg_w4_plan.h's functions, compiled by the host's compiler alone, for tests to call."""
import ctypes
import functools
import os
import subprocess
import tempfile

from fp8_grouped_gemm_tn_amd import build as kbuild

SOURCE = """
#include "kg_w4_plan.h"
extern "C" int set_outs(int all, int m0, int most) { return kg::w_set_outs(all, m0, most); }
extern "C" unsigned codes_left(int outs, int kbytes, int kb, int to) {
  return kg::w_codes_left(outs, kbytes, kb, to);
}
extern "C" int pieces(int nk) { return kg::w_pieces(nk); }
extern "C" void plan(long long M, int G, int N, int K, int cus, int kind, int group, int zp, long long* out) {
  const kg::WStream s = kg::w_stream(M, G, N, K, cus, kind, group, zp != 0);
  const kg::WTile t = kg::w_tile(M, G, N, K, cus, kind);
  const long long x[] = {kg::w_streams(s, t), s.rows, s.lds, s.tokens, s.scales, s.nj, s.waves, s.split, t.bt, t.bn, kg::kWLds};
  for (long long v : x) *out++ = v;
}
"""


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "w4_plan.so")
        subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-Wall", "-Werror",
                        "-I" + os.path.join(kbuild.PKG, "csrc"),
                        "-I" + os.path.join(kbuild.ROOT, "include"), "-x", "c++", "-", "-o", so],
                       input=SOURCE, text=True, check=True)
        L = ctypes.CDLL(so)
    L.codes_left.restype = ctypes.c_uint32
    return L


class Plan:
    """What a call takes: `streams`, and then rows, lds, tokens, scales (bytes), nj, waves, split;
    else a tile of bt x bn. limit: the LDS that a workgroup may ask for."""

    def __init__(self, M, G, N, K, kind, group, zp, cus=256):
        out = (ctypes.c_longlong * 11)()
        lib().plan(ctypes.c_longlong(M), G, N, K, cus, {"bf16": 0, "f32": 1, "e2m1": 2}[kind], group, zp, out)
        (self.streams, self.rows, self.lds, self.tokens, self.scales, self.nj, self.waves, self.split,
         self.bt, self.bn, self.limit) = out
