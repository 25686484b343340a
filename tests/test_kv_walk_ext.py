"""The attention kernels' work sharing with prefixes and first positions, their own arithmetic compiled for the host
(tests/csrc/kv_walk_ext.cu; CPU).  Signed overflow traps."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv_walk_ext") / "kv_walk_ext")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "--expt-relaxed-constexpr",
                    "-Xcompiler", "-fsanitize=signed-integer-overflow,-fsanitize-undefined-trap-on-error",
                    "-I", os.path.join(os.path.dirname(HERE), "include"), os.path.join(HERE, "csrc", "kv_walk_ext.cu"),
                    "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("mode", ["sorted", "wild"])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_shares_of_random_calls(walk, mode, seed):
    r = subprocess.run([walk, mode, str(seed), "300"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)
