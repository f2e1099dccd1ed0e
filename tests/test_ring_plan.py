"""The shared-memory ring's plan (csrc/row_ring.cuh), computed on the host alone.

The plan is ordinary host code: a small program around it prints it for groups of rows of
every kind, empty ones among them (rows without columns are valid and have no bytes).
"""
import shutil
import subprocess

import pytest

from nvfp4_precision_quantization_gb300 import build as lib_build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "row_ring.cuh"
using namespace nvfp4;
int main() {
  const long long bytes[] = {0, 2, 16, 50, 512, 8192, 10002, 65536, 98304, 131072, 262144};
  const int residents[] = {1, 2, 3, 8}, statics[] = {64, 9000, 40000};
  for (long long b : bytes)
    for (int tensors = 1; tensors <= 3; ++tensors)
      for (int any = 0; any < 2; ++any)
        for (int r : residents)
          for (int st : statics) {
            const RingPlan p = plan_ring(RingKernel{r, st}, tensors, b, any);
            printf("%lld %d %d %d %d %d %d %d %d\\n", b, tensors, any, r, st, p.ctas, p.g.stages,
                   p.g.tensor_bytes, p.g.stage_bytes);
          }
}
"""


def test_plan_holds_its_rows_or_is_empty(tmp_path):
    if shutil.which("nvcc") is None and shutil.which(lib_build.nvcc()) is None:
        pytest.skip("nvcc is not installed")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([lib_build.nvcc(), *lib_build.ARCH, "-std=c++17", "-w", "-I", lib_build.CSRC,
                    "-I", lib_build.INCLUDE, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.returncode
    lines = [tuple(map(int, line.split())) for line in run.stdout.splitlines()]
    assert len(lines) == 11 * 3 * 2 * 4 * 3
    for nbytes, tensors, any_, resident, static, ctas, stages, tensor, stage in lines:
        assert 0 <= ctas <= resident
        if nbytes == 0:
            assert ctas == 0
        if ctas == 0:
            continue
        assert 2 <= stages <= 8 and tensor % 128 == 0 and stage == tensors * tensor
        assert tensor >= nbytes + (128 if any_ else 0)
        # every CTA's ring, its static memory and 1 KB of the system's within an SM's 228 KB
        assert stages * stage + static <= 227 << 10
        assert ctas * (stages * stage + static + 1024) <= 228 << 10
