"""The key tiles that a prefill work item takes, up to the last position that 32 bits hold: the kernel's own index
functions, compiled for the host (no GPU needed) with traps where a signed sum overflows."""

import os
import random
import shutil
import subprocess

import pytest

from gemma_dual_geometry_gb300 import build as g4build

MAIN = r"""
#include <cuda_runtime.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "g4_internal.h"
#include "g4_tiles.h"

#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;

namespace g4 {
constexpr int kCausal = 0, kBidir = 1, kMods = 2, kBM = 128, kBN = 128;
@FUNCTIONS@
}  // namespace g4

using namespace g4;

int main() {
  int what, a0, a1, T, max_len, ring, window, own;
  while (scanf("%d %d %d %d %d %d %d %d", &what, &a0, &a1, &T, &max_len, &ring, &window, &own) == 8) {
    if (what == 0) {  // keys before a0 among the T from a1 on
      printf("%d\n", keys_before(a0, a1, T));
    } else if (what == 1) {  // tiles of the keys [a0, a1)
      TcItem w;
      tc_set_keys(w, a0, a1);
      printf("%d %d\n", w.kt_begin, w.ntiles);
    } else {  // all items of T tokens from q_start a0 on
      ModsTcArgs a = {};
      int begin = own ? a1 : 0, q_start = a0;
      a.q_start = &q_start;
      a.B = a.H = a.Hkv = 1;
      a.T = T;
      a.max_len = max_len;
      a.ring = ring;
      a.sliding = window > 0;
      a.window = window;
      std::vector<int> begins(T, begin);
      if (own) a.key_begin = begins.data();
      const int nqt = (T + kBM - 1) / kBM;
      for (int it = 0; it < nqt; ++it) {
        TcItem w;
        if (what == 2) {
          w = tc_item<1, kMods>(a, it, nqt);
          int lo = 0x7fffffff, hi = 0;
          for (int r = 0; r < kBM; ++r) {
            const int2 k = tc_row_keys(a, w, r);
            if (k.x < k.y) lo = min(lo, k.x), hi = max(hi, k.y);
          }
          tc_set_keys(w, hi == 0 ? 0 : lo, hi);
        } else {
          w = tc_item<1, kCausal>(static_cast<const PrefillTcArgs&>(a), it, nqt);
        }
        printf("%d %d %d ", w.kt_begin, w.ntiles, w.Lk);
      }
      printf("\n");
    }
  }
  return 0;
}
"""

LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    text = open(os.path.join(g4build.CSRC, "g4_prefill_tc.cuh")).read()
    functions = text[text.index("struct TcItem {"):text.index("// ---------------------------------------------------------------- MODS")]
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(g4build.nvcc_path()))), "include")
    tmp = tmp_path_factory.mktemp("tiles")
    src, exe = tmp / "tiles.cpp", tmp / "tiles"
    src.write_text("#include <vector>\n" + MAIN.replace("@FUNCTIONS@", functions))
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I", g4build.CSRC, "-I", include, str(src), "-o", str(exe)], check=True)

    def run(questions):
        text = "".join(" ".join(str(x) for x in (q + [0] * 8)[:8]) + "\n" for q in questions)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
        assert r.returncode == 0, "a signed sum overflowed"
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]

    return run


def near(rng):
    """A position near one of the range's ends or anywhere in it."""
    return rng.choice([rng.randrange(0, 400), LAST - rng.randrange(0, 400), rng.randrange(0, LAST + 1)])


def test_tiles_of_keys(ask):
    rng = random.Random(1)
    cases = [(0, 0), (0, 1), (127, 128), (128, 129), (0, LAST), (LAST - 1, LAST), (LAST - 1023, LAST), (LAST - 128, LAST - 127),
             (LAST - 127, LAST - 126)]
    cases += [tuple(sorted((near(rng), near(rng)))) for _ in range(500)]
    for (b, e), got in zip(cases, ask([[1, b, e] for b, e in cases])):
        assert got == [b // 128, -(-e // 128) - b // 128 if e > b else 0], (b, e)


def test_keys_of_a_tile_that_lie_before_an_end(ask):
    rng = random.Random(2)
    cases = [(LAST, LAST // 128 * 128, 128), (LAST, LAST // 64 * 64, 64), (5, LAST // 128 * 128, 128), (0, 0, 64), (64, 0, 64)]
    cases += [(near(rng), near(rng) // 64 * 64, rng.choice([64, 128])) for _ in range(500)]
    for (end, key, n), got in zip(cases, ask([[0, e, k, n] for e, k, n in cases])):
        assert got == [min(max(end - key, 0), n)], (end, key, n)


@pytest.mark.parametrize("own", [0, 1])
def test_items_at_the_last_positions_of_a_ring(ask, own):
    """Each item's tiles are those of the keys that its tokens see, for chunks that end with the last position."""
    rng = random.Random(3)
    cases = []
    for T, rows, window in ((1, 128, 8), (80, 1024, 40), (128, 256, 128), (300, 1024, 500), (129, 384, 256)):
        for start in (0, 1000, LAST - T - 300, LAST - T - 128, LAST - T - 1, LAST - T, LAST - T - rng.randrange(0, 128)):
            cases.append((T, rows, window, start, max(0, start + T - rows + rng.randrange(-5, rows // 2))))
    got = ask([[2, start, begin, T, rows, 1, window, own] for T, rows, window, start, begin in cases])
    plain = ask([[3, start, begin, T, rows, 1, window, 0] for T, rows, window, start, begin in cases])
    for (T, rows, window, start, begin), items, causal in zip(cases, got, plain):
        n = -(-T // 128)
        held = start + T
        for i in range(n):
            first, last = start + 128 * (n - 1 - i), min(start + T, start + 128 * (n - i)) - 1
            lo = max(begin if own else first - window + 1, 0, held - rows)
            want = [lo // 128, last // 128 + 1 - lo // 128] if lo <= last else [0, 0]
            assert items[3 * i:3 * i + 2] == want, (T, rows, window, start, i)
            lo = max(first - window + 1, 0)
            assert causal[3 * i:3 * i + 2] == [lo // 128, last // 128 + 1 - lo // 128], (T, rows, window, start, i)
