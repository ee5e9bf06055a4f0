"""The check of one access that the bounds-checked build makes (csrc/s4_extents.h), compiled for the CPU: what it
lets pass, and that it finds accesses outside of an array, between its rows, of the wrong kind and misaligned ones."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <stdio.h>
#include <initializer_list>
#include "s4_extents.h"
struct Rows { const void* p; long long batch, row; };
static int failed = 0;
static void expect(bool got, bool want, int line) {
  if (got != want) { failed = 1; printf("line %d: %d\n", line, got); }
}
#define EXPECT(got, want) expect(got, want, __LINE__)
int main() {
  using namespace s4impl;
  const unsigned long long A = 0x100000;
  const auto at = [](unsigned long long v) { return (const void*)v; };
  const auto ok = [&](const Extents& x, unsigned long long p, long long bytes, int align, bool write) {
    return access_ok(x.list, x.n, p, bytes, align, write);
  };
  {  // one dense array of 10 floats, read only
    Extents x{};
    x.in(at(A), 4, 10);
    x.in(nullptr, 4, 10);
    EXPECT(x.n == 1, true);
    EXPECT(ok(x, A, 16, 16, false), true);
    EXPECT(ok(x, A + 36, 4, 4, false), true);
    EXPECT(ok(x, A + 32, 16, 16, false), false);  // its last pack is not whole
    EXPECT(ok(x, A + 40, 4, 4, false), false);
    EXPECT(ok(x, A - 4, 4, 4, false), false);
    EXPECT(ok(x, A, 4, 4, true), false);          // not written
    EXPECT(ok(x, A + 8, 16, 16, false), false);   // misaligned
    EXPECT(ok(x, A + 8, 8, 8, false), true);
  }
  {  // [2][3] rows of 8 of 20 bfloat16 channels, 100 elements from sequence to sequence
    Extents x{};
    x.out_rows(Rows{at(A), 100, 20}, 2, 2, 3, 8);
    for (int b = 0; b < 2; ++b)
      for (int t = 0; t < 3; ++t) {
        const unsigned long long r = A + 2 * (100 * b + 20 * t);
        EXPECT(ok(x, r, 16, 4, true), true);
        EXPECT(ok(x, r + 14, 2, 2, true), true);
        EXPECT(ok(x, r + 16, 2, 2, true), false);  // the channels of another array
        EXPECT(ok(x, r - 2, 2, 2, true), false);
      }
    EXPECT(ok(x, A + 2 * 60, 2, 2, true), false);    // a fourth token
    EXPECT(ok(x, A + 2 * 200, 2, 2, true), false);   // a third sequence
  }
  {  // tokens outermost, sequences inside
    Extents x{};
    x.in_rows(Rows{at(A), 8, 64}, 4, 4, 5, 8);
    EXPECT(ok(x, A + 4 * (64 * 4 + 8 * 3), 32, 16, false), true);
    EXPECT(ok(x, A + 4 * (64 * 4 + 8 * 4), 4, 4, false), false);
  }
  {  // groups of states inside rows; a broadcast row; one sequence with any stride
    Extents x{};
    x.add(at(A), 4, true, false, 5, 2, 1000, 3, 100, 4, 10);
    EXPECT(ok(x, A + 4 * (1000 + 200 + 30 + 4), 4, 4, false), true);
    EXPECT(ok(x, A + 4 * (1000 + 200 + 30 + 5), 4, 4, false), false);
    EXPECT(ok(x, A + 4 * (1000 + 200 + 40), 4, 4, false), false);
    Extents y{};
    y.in_rows(Rows{at(A), 0, 0}, 4, 7, 9, 6);
    y.in_rows(Rows{at(A + 4096), 3, 6}, 4, 1, 9, 6);
    EXPECT(ok(y, A + 20, 4, 4, false), true);
    EXPECT(ok(y, A + 24, 4, 4, false), false);
    EXPECT(ok(y, A + 4096 + 4 * 53, 4, 4, false), true);
    EXPECT(ok(y, A + 4096 + 4 * 54, 4, 4, false), false);
  }
  {  // far rows: offsets beyond 32 bits
    Extents x{};
    const long long far = (1ll << 31) + 8;
    x.in_rows(Rows{at(A), far, 64}, 2, 2, 3, 64);
    EXPECT(ok(x, A + 2 * (far + 191), 2, 2, false), true);
    EXPECT(ok(x, A + 2 * (far + 192), 2, 2, false), false);
  }
  {  // rows of H (N + 2) sums that are stored in words of 16 bytes: every second one of an odd H is misaligned
    // unless the rows are padded
    const long long H = 333, N = 16, dense = H * (N + 2), padded = (dense + 3) / 4 * 4;
    for (long long pitch : {dense, padded}) {
      Extents x{};
      x.add(at(A), 4, true, true, dense, 4, pitch);
      for (int r = 0; r < 4; ++r) EXPECT(ok(x, A + 4 * r * pitch, 16, 16, true), pitch == padded || r % 2 == 0);
    }
  }
  return failed;
}
"""


def test_the_check_of_an_access(tmp_path):
    src, exe = tmp_path / "extents.cpp", tmp_path / "extents"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "structured_state_space_gb300", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

