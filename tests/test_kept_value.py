"""A value that the library asks the runtime for once: a failure of the first query is not kept (no GPU: the query is a
stand-in, compiled with the library's header)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "cba_kept.cuh"
int main() {
    std::atomic<int> kept{0};
    int asked = 0, v = -1;
    auto fails = [&](int *) { ++asked; return cudaErrorMemoryAllocation; };
    auto none = [&](int *n) { ++asked; *n = 0; return cudaSuccess; };
    auto gives = [&](int *n) { ++asked; *n = 3; return cudaSuccess; };
    if (cba::kept_value(kept, &v, fails) != cudaErrorMemoryAllocation || v != -1) return 1;       // the error itself
    if (cba::kept_value(kept, &v, none) != cudaErrorInvalidConfiguration || v != -1) return 2;
    if (cba::kept_value(kept, &v, gives) != cudaSuccess || v != 3 || asked != 3) return 3;        // asked again
    v = 0;
    if (cba::kept_value(kept, &v, fails) != cudaSuccess || v != 3 || asked != 3) return 4;        // kept
    return 0;
}
"""


def test_a_failed_query_is_asked_again(tmp_path):
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(cuda, "include")):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "kept.cpp", tmp_path / "kept"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(cuda, "include"), "-I",
                    os.path.join(ROOT, "activation_backward_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_layer_norm_keeps_no_static_result_of_a_query():
    """Every function-local static of the launch code is an atomic."""
    with open(os.path.join(ROOT, "activation_backward_gb300", "csrc", "cba_layernorm.cu")) as f:
        lines = [s.strip() for s in f if s.startswith("    static ")]
    assert lines and all("std::atomic" in s for s in lines), lines
