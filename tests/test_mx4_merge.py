"""Which blocks the widest form of the product over microscaled 4-bit weights takes together (mx_merge in
csrc/mol_internal.h, compiled with the host compiler): each size that it takes together is one that the launch rule sends to
that form, for the same rows of x."""
import os
import subprocess

from tests import conftest

SRC = r'''
#include <cstdio>
#include <cstdint>
#include <algorithm>
#include "mol_internal.h"
int main() {
  for (int rows : {mol::kMxRowsBf16, mol::kMxRowsF32, mol::kMxRowsCodes})
    for (long long BM = 1; BM <= 260; ++BM) {
      bool wide = false;
      for (long long E : {1, 8, 128})
        for (long long N : {64, 1536, 12000})
          for (long long pairs = 1; pairs < (1 << 22); pairs = pairs * 3 / 2 + 1)
            wide |= mol::mx_form(pairs, E, N, BM, rows) == mol::kMxWide;
      std::printf("%d %lld %d %d\n", rows, BM, mol::mx_merge(BM, rows), (int)wide);
    }
}
'''


def test_blocks_taken_together_reach_the_form_that_takes_them(tmp_path):
    src, exe = tmp_path / "merge.cpp", tmp_path / "merge"
    src.write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(conftest.ROOT, "virtual_expert_routed_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], text=True, capture_output=True, check=True).stdout
    rows = [tuple(map(int, ln.split())) for ln in out.splitlines()]
    assert all(wide for _, _, merge, wide in rows if merge > 1)
    assert {(r, bm, merge) for r, bm, merge, _ in rows if merge > 1} == {(r, bm, 128 // bm) for r in (0, 2) for bm in (16, 32, 64)}
