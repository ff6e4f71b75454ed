"""Launch grids on the CPU: a dimension of a grid holds fewer than 2^32
threads, and every group has its workgroup."""
import os
import subprocess

import pytest

from selective_state_space_25_amd import build

# workgroups of 256 threads: one; at and past a dimension's first 2^20; dq of
# batch 1, L 2^20, 32 groups of 128 (2^32 elements); the largest dropout
COUNTS = [1, 5, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, (1 << 32) // 256, (1 << 32) // 256 + 1, (1 << 35) - 3]


@pytest.fixture(scope="module")
def grids(tmp_path_factory):
    d = tmp_path_factory.mktemp("grids")
    src = d / "grids.cpp"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "io.hpp"\n'
                   "int main(int n, char** v) {\n"
                   "    for (int i = 1; i < n; ++i) {\n"
                   "        const dim3 g = selscan::io::groups(std::strtoll(v[i], nullptr, 10));\n"
                   '        std::printf("%u %u %u\\n", g.x, g.y, g.z);\n'
                   "    }\n}\n")
    subprocess.run([build.hipcc(), "-x", "hip", "--cuda-host-only", "-O1", "-std=c++17", "-I", build.INCLUDE, "-I",
                    build.CSRC, "-c", str(src), "-o", str(d / "grids.o")], check=True, capture_output=True)
    subprocess.run([build.hipcc(), str(d / "grids.o"), "-o", str(d / "grids")], check=True, capture_output=True)
    out = subprocess.run([str(d / "grids")] + [str(n) for n in COUNTS], check=True, capture_output=True, text=True)
    return dict(zip(COUNTS, (tuple(map(int, l.split())) for l in out.stdout.splitlines())))


@pytest.mark.parametrize("n", COUNTS)
def test_groups(grids, n):
    x, y, z = grids[n]
    assert x * 256 < 1 << 32 and y < 1 << 16 and z == 1
    assert n <= x * y < n + x


def test_group_sum_is_launched_over_groups():
    """The sum over a group's heads has a thread for each element of dq, which can be 2^32 of them and more."""
    src = open(os.path.join(build.CSRC, "delta_bwd.hip")).read()
    at = src.index("hipLaunchKernelGGL((delta_group_kernel")
    assert "io::groups(" in src[at:src.index(";", at)]
    kernel = src.index("void delta_group_kernel")
    assert "io::group_id()" in src[kernel:kernel + 400]
