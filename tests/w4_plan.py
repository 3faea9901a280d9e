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
