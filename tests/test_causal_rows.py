"""CPU replay of a causal convolution worker's way through its rows (tests/replay/causal_rows_replay.cu)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rows(tmp_path):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if not nvcc:
        pytest.skip("nvcc not available")
    out = str(tmp_path / "replay")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-o", out,
                        os.path.join(HERE, "replay", "causal_rows_replay.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    for seed in ("1", "2"):
        r = subprocess.run([out, seed, "400"], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "errors: 0" in r.stdout, r.stdout[-2000:]
