"""Positions of the window kernels at the largest sizes that a call may have, under the
host's check for signed overflow (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "window_launch.h"
int main() {
    const int most = 2147483647 - 4095;   // keys of a sequence
    const int keys[] = {0, 1, 63, 1 << 30, most - 64, most - 1}, windows[] = {1, 100, 1 << 30, most};
    for (int key : keys)
        for (int window : windows)
            for (long long from : {(long long)key, (long long)key + 1, (long long)key + window - 1, (long long)key + window,
                                   (long long)key + window + 1, (long long)most - 1}) {
                if (from < key || from >= most) continue;
                const long long want = (long long)key + window - from;
                if (kda::positions_in_window(key, window, (int)from) != (want > 0 ? want : 0)) {
                    printf("key %d, window %d, from %lld\n", key, window, from);
                    return 1;
                }
            }
    return 0;
}
"""


def test_positions_in_window(tmp_path):
    include = "/opt/rocm/include"
    if not shutil.which("g++") or not os.path.exists(os.path.join(include, "hip", "hip_runtime_api.h")):
        pytest.skip("no g++ or no HIP headers")
    src, exe = tmp_path / "positions.cpp", tmp_path / "positions"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-isystem", include, "-I",
                        os.path.join(ROOT, "gated_delta_rule_prefill_amd", "csrc"), "-fsanitize=signed-integer-overflow",
                        "-fno-sanitize-recover=all", "-o", str(exe), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
