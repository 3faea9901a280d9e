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


ROW_UNITS = """
using namespace kg;
constexpr bool has_unit(const RowShape& s, int64_t id, int sub, int lane, int64_t token, int unit) {
  int64_t t = -1;
  int c = -1;
  return unit_of(s, id, 256 / s.lanes, sub, lane, &t, &c) && t == token && c == unit;
}
constexpr bool none(const RowShape& s, int64_t id, int sub) {
  int64_t t = -1;
  int c = -1;
  return !unit_of(s, id, 256 / s.lanes, sub, 0, &t, &c);
}
// 48 units to a row: 3 runs of 16, 16 runs to a workgroup, and as many runs as there may be (the
// last one's number is 2^32 - 260). 2^28 workgroups fill 32 lines of 2^23.
constexpr int64_t T = (((int64_t)1 << 32) - 259) / 3;
constexpr RowShape wide = {T, T, 1, 384, 16, 3, (T * 3 + 15) / 16};
static_assert(T * 3 == ((int64_t)1 << 32) - 259 && wide.groups == ((int64_t)1 << 28) - 16, "");
static_assert(has_unit(wide, 0, 0, 5, 0, 5) && has_unit(wide, 0, 4, 15, 1, 31), "");
static_assert(has_unit(wide, wide.groups - 1, 12, 1, T - 1, 33) && none(wide, wide.groups - 1, 13), "");
// the workgroups past them, whose runs' numbers pass 2^32 from the second on
static_assert(none(wide, wide.groups, 0) && none(wide, wide.groups + 15, 15), "");
static_assert(none(wide, wide.groups + 16, 0) && none(wide, wide.groups + 16, 15), "");
static_assert(none(wide, wide.groups + kGroupsX - 1, 7), "");
// one run to a token: its number may pass 2^32
constexpr RowShape narrow = {(int64_t)1 << 31, (int64_t)1 << 31, 1, 8, 16, 1, (int64_t)1 << 27};
static_assert(has_unit(narrow, narrow.groups - 1, 15, 0, narrow.T - 1, 0), "");
static_assert(none(narrow, narrow.groups, 0) && none(narrow, (int64_t)1 << 28, 3), "");
"""


def test_row_copies_past_their_last_workgroup(tmp_path):
    """Workgroups that only fill up a launch's last line have no unit, also where the number of
    their run passes 32 bits."""
    ok, messages = compiles(tmp_path, "kg_route.hip", ROW_UNITS)
    assert ok, messages
