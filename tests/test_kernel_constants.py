"""What the kernels' sources compute at compile time, checked by the compiler's front end on the
host's side: nothing is run, and an index out of range is no constant expression."""
import os
import subprocess

from fp8_grouped_gemm_tn_amd import build as kbuild

CSRC = os.path.join(kbuild.PKG, "csrc")


def compiles(tmp_path, source, checks):
    """(the front end takes `checks` behind csrc/`source`, its messages)."""
    tu = tmp_path / "checks.hip"
    tu.write_text(f'#include "{os.path.join(CSRC, source)}"\n{checks}\n')
    flags = [f for f in kbuild.FLAGS if f not in ("-fPIC", "-O3")]
    r = subprocess.run([kbuild.HIPCC] + flags + ["--offload-host-only", "-fsyntax-only", str(tu)],
                       capture_output=True, text=True)
    return r.returncode == 0, r.stderr


FPROP_SUMS = """
using namespace kg;
// The forward product's walk over a block's partial sums: the one of MFMA u - LAG is added after
// MFMA u, the last LAG ones behind the loop. Each once, behind its own MFMA, before its place in
// the ring of LAG + 1 is written again.
template <class C>
constexpr bool once() {
  int added[C::SUMS] = {}, held[C::LAG + 1] = {};
  for (int u = 0; u < C::SUMS; ++u) {
    held[u % (C::LAG + 1)] = u;
    if (u >= C::LAG) {
      if (held[(u - C::LAG) % (C::LAG + 1)] != u - C::LAG) return false;
      ++added[u - C::LAG];
    }
  }
  for (int u = C::SUMS - C::LAG; u < C::SUMS; ++u) {
    if (held[u % (C::LAG + 1)] != u) return false;
    ++added[u];
  }
  for (int n : added)
    if (n != 1) return false;
  return true;
}
static_assert(once<FCfg<256, 256, 4, 1>>() && once<FCfg<128, 256, 2, 1>>(), "");
static_assert(once<FCfg<128, 128, 4, 1>>() && once<FCfg<128, 128, 4, 2>>(), "");
static_assert(once<FCfg<64, 128, 2, 2>>() && once<FCfg<64, 128, 2, 2, true>>(), "");
static_assert(once<FCfg<64, 64, 4, 2>>(), "");
"""


def test_partial_sums_of_every_tile(tmp_path):
    ok, messages = compiles(tmp_path, "kg_fprop.hip", FPROP_SUMS)
    assert ok, messages


def test_a_lag_that_passes_the_sums_is_refused(tmp_path):
    """The check above sees what it is for."""
    wrong = FPROP_SUMS + "struct Late : FCfg<64, 64, 4, 2> { static constexpr int LAG = 3; };\n" \
        'static_assert(once<Late>(), "");\n'
    ok, messages = compiles(tmp_path, "kg_fprop.hip", wrong)
    assert not ok and "constant expression" in messages
