"""The work sharing of the attention kernels over the 4-bit cache, with the
kernels' own arithmetic compiled for the host (tests/csrc/kv_walk.cu; CPU): every
tile of every item lies in one share, a 128-row tile takes no tile that its share
does not hold, and no token that a row sees is left out.  Signed overflow traps."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv_walk") / "kv_walk")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17",
                    "--expt-relaxed-constexpr", "-Xcompiler",
                    "-fsanitize=signed-integer-overflow,-fsanitize-undefined-trap-on-error",
                    "-I", os.path.join(os.path.dirname(HERE), "include"),
                    os.path.join(HERE, "csrc", "kv_walk.cu"), "-o", exe], check=True)
    return exe


def _run(walk, mode, seed, calls):
    r = subprocess.run([walk, mode, str(seed), str(calls)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)


@pytest.mark.parametrize("mode", ["prompts", "few", "wide_windows", "long_caches", "more_rows"])
@pytest.mark.parametrize("seed", [1, 2])
def test_shares_of_random_calls(walk, mode, seed):
    _run(walk, mode, seed, 400)
