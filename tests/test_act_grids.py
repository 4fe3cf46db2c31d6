"""The grids of the activation entry points over long inputs (CPU, no device call):
tests/native/act_grid_check.cpp records the launches that the library's host code
makes, through stand-ins for the HIP runtime's launch calls."""
import os
import subprocess

import pytest

from conftest import ROOT

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_launches_stay_within_hip_and_cover_every_row(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    csrc = os.path.join(ROOT, "zero_sharded_mixed_bucketed_amd", "csrc")
    exe = str(tmp_path / "act_grid_check")
    srcs = [os.path.join(ROOT, "tests", "native", "act_grid_check.cpp")]
    srcs += [os.path.join(csrc, f) for f in ("act_api.hip", "block_norm.hip", "ckpt_store.hip",
                                             "ckpt_weight_grad.hip")]
    objs = []
    for s in srcs:
        objs.append(str(tmp_path / (os.path.basename(s) + ".o")))
        r = subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1",
                            "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                            "-x", "hip", "-c", s, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    # without their device code, which nothing here touches
    r = subprocess.run([HIPCC, *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "act grid check ok" in r.stdout
