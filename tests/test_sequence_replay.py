"""CPU replays of the selective scan's launch plans and of the causal convolution's work split (tests/replay/scan_plan_replay.cu,
tests/replay/causal_walk_replay.cu)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def replays(tmp_path_factory):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if not nvcc:
        pytest.skip("nvcc not available")
    out = tmp_path_factory.mktemp("replay")
    for name in ("scan_plan_replay", "causal_walk_replay"):
        r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-o",
                            str(out / name), os.path.join(HERE, "replay", name + ".cu")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    return out


@pytest.mark.parametrize("name", ["scan_plan_replay", "causal_walk_replay"])
@pytest.mark.parametrize("seed", [1, 2])
def test_plans(replays, name, seed):
    r = subprocess.run([str(replays / name), str(seed), "4000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "errors: 0" in r.stdout, r.stdout[-2000:]
