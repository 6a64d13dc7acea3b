"""Decisions of the attention that are plain functions of integers, compiled from
the kernels' own header and run on the CPU."""
import os
import subprocess

import numpy as np
import pytest

from masking_tm_affine_gb300 import build

PROGRAM = r"""
#include "tm_kv4_attn.cuh"
#include <cstdio>

int main()
{
    int first, count, grid;
    while (std::scanf("%d %d %d", &first, &count, &grid) == 3)
        std::printf("%d\n", libtm::job_in_grid(first, count, grid) ? 1 : 0);
    return 0;
}
"""


@pytest.fixture(scope="module")
def job_in_grid():
    work = os.path.join(build.BUILD, "host_check")  # the package's (ignored) build folder
    os.makedirs(work, exist_ok=True)
    src, exe = os.path.join(work, "jobs.cu"), os.path.join(work, "jobs")
    with open(src, "w") as f:
        f.write(PROGRAM)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I" + build.CSRC, "-I" + build.INCLUDE, src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(rows):
        out = subprocess.run([exe], input="\n".join("%d %d %d" % r for r in rows), capture_output=True, text=True, timeout=60)
        assert out.returncode == 0, out.stderr
        return [bool(int(x)) for x in out.stdout.split()]
    return ask


def test_a_job_that_nobody_noted_is_not_followed(job_in_grid):
    """The join reads partial outputs of blocks first .. first + count - 1: none outside the launch, whatever a
    block that gave up has left in the workspace."""
    rng = np.random.default_rng(0)
    most, least, nan = 2**31 - 1, -2**31, 0x7FC00000
    edge = [0, 1, 2, 151, 152, 153, 607, 608, 609, -1, most, most - 1, least, least + 1, nan, -1515870811]
    rows = [(f, c, g) for f in edge for c in edge for g in (1, 152, 608)]
    rows += [(int(f), int(c), 608) for f, c in rng.integers(least, most, (2000, 2), dtype=np.int64, endpoint=True)]
    rows += [(int(f), int(c), 152) for f, c in rng.integers(-4, 160, (2000, 2))]
    assert job_in_grid(rows) == [f >= 0 and c >= 1 and f + c <= g for f, c, g in rows]
