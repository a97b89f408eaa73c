"""CPU replay of the cluster Newton-Schulz kernel's shared-memory plan (tests/replay/newton_small_replay.cu)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if not nvcc:
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("replay") / "newton_small_replay")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-o", exe,
                        os.path.join(HERE, "replay", "newton_small_replay.cu"), "-lcuda"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


# (first m, last m, step of n): every m with a stride of n that meets odd and even sizes, and
# the sizes about whole chunks of 64 closely
@pytest.mark.parametrize("span", [(1, 64, 13), (65, 128, 13), (33, 34, 1), (95, 96, 1), (128, 128, 1)])
def test_cluster_plan(replay, span):
    r = subprocess.run([replay, *map(str, span)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "errors: 0" in r.stdout, r.stdout[-2000:]
