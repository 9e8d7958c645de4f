"""The launch rule of the weight streams (stream_items in csrc/mol_internal.h, compiled with the host compiler)
takes the form that each case of stream_cases.py is there to test, so that a change of the rule cannot move
those tests to another kernel unseen."""
import os
import subprocess

from tests import conftest, stream_cases as sc

SRC = r'''
#include <cstdio>
#include <cstdint>
#include <algorithm>
#include "mol_internal.h"
int main() {
  long long m, p, rows, bytes;
  while (std::scanf("%lld %lld %lld %lld", &m, &p, &rows, &bytes) == 4) {
    const mol::StreamItems it = mol::stream_items(m, p, rows, bytes);
    std::printf("%d %d\n", it.split ? 1 : 0, it.tiles);
  }
}
'''


def forms(tmp_path, asked):
    src, exe = tmp_path / "forms.cpp", tmp_path / "forms"
    src.write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(conftest.ROOT, "virtual_expert_routed_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, a)) for a in asked), text=True,
                       capture_output=True, check=True)
    return [tuple(map(int, ln.split())) for ln in r.stdout.splitlines()]


def test_the_cases_take_the_forms_they_name(tmp_path):
    asked, want = [], []
    for E, N, block_m, K, form in sc.PRODUCT:
        pairs = len(sc.product_pairs(E))
        blocks = min(pairs, E + pairs // block_m)  # as mol_moe_gemm_q4 counts them
        for k in K.values():
            asked.append((blocks, pairs, N, k // 2))
            want.append(form)
    layers = [(*case, len(sc.product_pairs(case[2])), case[2]) for case in sc.LAYER]
    assert all(pairs > E for *_, pairs, E in layers)  # by expert
    layers += [(dtype, group, 130, H, I, gu, dn, 96, 96) for dtype, group, H, I, gu, dn in sc.BY_PAIR]
    for dtype, group, _, H, I, gu, dn, pairs, matrices in layers:
        def row_bytes(k):
            return k // 2 if group else k * (2 if dtype == "bf16" else 4)
        asked += [(matrices, pairs, 2 * I, row_bytes(H)), (matrices, pairs, H, row_bytes(I))]
        want += [gu, dn]
    got = forms(tmp_path, asked)
    assert got == want, [(a, g, w) for a, g, w in zip(asked, got, want) if g != w]
