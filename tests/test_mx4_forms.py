"""The launch rule of the product over microscaled 4-bit weights (mx_form in csrc/mol_internal.h, compiled with the host
compiler) takes the form that each case of mx4_cases.py is there to test."""
import os
import subprocess

from tests import conftest, mx4_cases as mc

SRC = r'''
#include <cstdio>
#include <cstdint>
#include <algorithm>
#include "mol_internal.h"
int main() {
  long long pairs, E, N, BM, rows;
  while (std::scanf("%lld %lld %lld %lld %lld", &pairs, &E, &N, &BM, &rows) == 5)
    std::printf("%d\n", mol::mx_form(pairs, E, N, BM, (int)rows));
}
'''


def test_the_cases_take_the_forms_they_name(tmp_path):
    src, exe = tmp_path / "forms.cpp", tmp_path / "forms"
    src.write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(conftest.ROOT, "virtual_expert_routed_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    asked = []
    for x, M, E, topk, K, N, block_m, form in mc.FORMS + mc.POPULAR:
        asked.append((M * topk, E, N, block_m, {"bf16": 0, "f32": 1, "codes": 2}[x]))
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, a)) for a in asked), text=True, capture_output=True,
                       check=True)
    got = [int(ln) for ln in r.stdout.splitlines()]
    cases = mc.FORMS + mc.POPULAR
    assert got == [c[-1] for c in cases], [(c, g) for c, g in zip(cases, got) if c[-1] != g]
    assert {(c[0], c[-1]) for c in mc.FORMS} == {(x, f) for x in ("bf16", "codes", "f32") for f in (mc.NARROW, mc.WIDE)} | {
        ("f32", mc.SPLIT), ("bf16", mc.SPREAD), ("codes", mc.SPREAD)}
