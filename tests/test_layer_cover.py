"""Which kernels of the feed-forward block the GPU tests' sizes reach, from the
library's own host code built for the CPU (tests/host_check/layer_cover.cpp): a
change of the plan that takes a kernel out of the tests' reach fails here."""

import itertools
import os
import shutil
import subprocess

import pytest

from tests.layer_sizes import TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = [os.path.join(ROOT, "newton_schulz_09_amd", "csrc", "layer_api.hip"),
           os.path.join(ROOT, "tests", "host_check", "layer_cover.cpp")]


def test_sizes_reach_every_kernel(tmp_path):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc is not available")
    objs = []
    for src in SOURCES:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-c", src, "-o", objs[-1]],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    exe = str(tmp_path / "layer_cover")
    r = subprocess.run([HIPCC, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe, *(str(n) for size in TILES for n in size)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    got = {tuple(line.split()[3:]) for line in r.stdout.splitlines()}
    want = set(itertools.product(("gated", "plain", "hidden", "input", "weights"), ("128", "256"), ("whole", "split", "mixed")))
    assert got == want, sorted(want - got)
    assert all(n % 16 and width % 64 and hidden % 64 for n, width, hidden in TILES if width != 1600)
