"""The wait limits of the attention kernels (no GPU): csa_attn_limits.h compiled for the host."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_indexer_csa_gb300", "csrc")
STEP_NS = 1400  # of one block of 128 rows and 128 keys at full clock


@pytest.fixture(scope="module")
def limits(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("limits")
    src, lib = d / "limits.cc", d / "limits.so"
    src.write_text('#include "csa_attn_limits.h"\nextern "C" {\n'
                   "unsigned long long by_keys(long long tk) { return csa::attn_wait_ns(csa::attn_steps_keys(tk)); }\n"
                   "unsigned long long by_rows(long long t, long long q) { return csa::attn_wait_ns(csa::attn_steps_rows(t, q)); }\n"
                   "}\n")
    subprocess.run([cc, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    for f, n in ((so.by_keys, 1), (so.by_rows, 2)):
        f.restype, f.argtypes = ctypes.c_uint64, [ctypes.c_int64] * n
    return so


@pytest.mark.parametrize("tokens,heads", [(0, 1), (1, 128), (8192, 8), (1_000_000, 8), (1_500_000, 128), (4_000_000, 128)])
def test_the_longest_item_fits_several_times(limits, tokens, heads):
    """An item of dk and dv walks all rows of a sequence, 128/heads tokens a step."""
    steps = -(-tokens // (128 // heads))
    assert limits.by_rows(tokens, 128 // heads) >= max(2e9, 10 * steps * STEP_NS)
    assert limits.by_keys(tokens) >= max(2e9, 10 * -(-tokens // 128) * STEP_NS)


def test_waits_stay_short_for_ordinary_calls(limits):
    assert limits.by_keys(131072) < 2.1e9 and limits.by_rows(16384, 16) < 2.1e9


def test_every_launch_takes_its_limit_from_its_steps():
    for name, launches in (("csa_attn_fwd.cu", 1), ("csa_attn_bwd.cu", 2)):
        text = open(os.path.join(CSRC, name)).read()
        assert len(re.findall(r"f\.wait_ns = attn_wait_ns\(attn_steps_(?:keys|rows)\(", text)) == launches
        assert len(re.findall(r"f\.wait_ns =", text)) == launches


def test_copies_in_flight_are_waited_for_wherever_a_cta_gives_up(tmp_path):
    """A model of the producer's rings: random tiles, some of them mended, given up after any of them.  What drain()
    asks for is, for each stage that a copy was started into, the barrier and the parity of the phase that its last
    copy completes."""
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    src = tmp_path / "copies.cc"
    src.write_text(r"""
#include <cstdio>
#include <cstdlib>
#include "csa_attn_limits.h"
int main() {
  srand(7);
  for (int round = 0; round < 2000; ++round) {
    const int stages = 1 + rand() % 9, tiles = rand() % 60;
    csa::Copies c;
    int ring[9] = {}, other[9] = {};            // phases begun on a stage's two barriers
    int want[9], parity[9];                     // -1: no copy; 0: ring barrier; 1: the other
    for (int s = 0; s < 9; ++s) want[s] = -1;
    for (int i = 0; i < tiles; ++i) {
      const int s = i % stages;
      const bool mend = rand() % 3 == 0;
      c.start(s, mend, (i / stages) & 1);
      want[s] = mend;
      parity[s] = (mend ? other[s]++ : ring[s]) & 1;
      ++ring[s];                                // completed by the copy, or by who mends the tile
    }
    int asked = 0, all = 0;
    bool good = true;
    for (int s = 0; s < 9; ++s) all += want[s] >= 0;
    c.drain([&](int s, bool mend, unsigned p) {
      ++asked;
      good = good && s < 9 && want[s] == int(mend) && parity[s] == int(p);
    });
    if (!good || asked != all) return printf("round %d\n", round), 1;
  }
  return 0;
}
""")
    exe = tmp_path / "copies"
    subprocess.run([cc, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True)
