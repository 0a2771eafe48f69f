"""The grids of the language-model kernels and where their partial outputs lie,
on the CPU (tests/host_check/lm_grid.cpp)."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_grids_stay_within_the_limits(tmp_path):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc is not available")
    exe = str(tmp_path / "lm_grid")
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1",
                        os.path.join(ROOT, "tests", "host_check", "lm_grid.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "grids ok" in r.stdout, r.stdout + r.stderr


def test_every_launch_that_grows_with_the_rows_uses_them():
    """Launches with another grid: the split kernel below 257 workgroups, and the
    norm's, which are bounded where they are planned."""
    for name, others in (("attn_fwd", 1), ("attn_bwd", 0), ("embed", 2), ("qk_norm", 2)):
        text = open(os.path.join(ROOT, "newton_schulz_09_amd", "csrc", name + ".hip"), encoding="utf-8").read()
        launches = re.findall(r"<<<(\w+)", text)
        assert len([x for x in launches if x != "long_grid"]) == others, (name, launches)
        assert name != "embed" or launches.count("sorts") == 2  # made by long_grid
        assert name == "qk_norm" or "blockIdx.x" not in text  # places come from block_place
