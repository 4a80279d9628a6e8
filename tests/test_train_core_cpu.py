"""Index arithmetic of the training operators' kernels, compiled for the host."""
import os
import subprocess

import pytest

from adamw_optimizer_step_tensor_amd import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

UNLIMITED = r"""
#include <stdio.h>
#include "gemm.h"
// Loads without a limit read whole 16-byte chunks of kCols rows, so another row has to follow those that they read.
int main()
{
    using namespace train;
    for (int depth = 0; depth <= 4100; ++depth)
        for (int step = 0; step <= last_inside(depth); step += kStages)
            for (int s = 0; s < kStages; ++s) {
                const int tile = step + s + kStages - 1;  // what run_step's load of stage s brings
                if ((tile + 1) * kStep >= depth) return printf("depth %d: tile %d is the last\n", depth, tile), 1;
            }
    // and no more is given up than the last tile: the next kStages steps would reach it
    for (int depth = 1; depth <= 4100; ++depth)
        if ((last_inside(depth) + 1 + 2 * kStages - 1) * kStep < depth) return printf("depth %d\n", depth), 2;
    return 0;
}
"""


@pytest.fixture(scope="module")
def compile_host(tmp_path_factory):
    def compiled(text):
        at = tmp_path_factory.mktemp("host")
        source, exe = at / "probe.hip", at / "probe"
        source.write_text(text)
        subprocess.run([lib_build.hipcc(), "--cuda-host-only", "-std=c++17", "-O1", "-Wno-unused-command-line-argument",
                        f"-I{lib_build.INCLUDE}", f"-I{os.path.join(lib_build.PKG, 'csrc')}", str(source), "-o", str(exe)],
                       check=True)
        return str(exe)

    return compiled


def test_unlimited_loads_stay_before_the_last_tile(compile_host):
    run = subprocess.run([compile_host(UNLIMITED)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout
