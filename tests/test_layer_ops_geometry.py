"""The launch geometry of the convolution and the selective scan at sizes near
the limits, on the CPU."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"
SOURCES = [os.path.join(ROOT, *p.split("/")) for p in (
    "mamba_chunked_ssd_amd/csrc/ssd_api.cpp", "mamba_chunked_ssd_amd/csrc/ssd_bwd.cpp",
    "mamba_chunked_ssd_amd/csrc/ssd_ops.cpp", "tests/host/stub_launch.cpp", "tests/host/stub_ops_launch.cpp",
    "tests/host/geometry_driver.cpp")]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="needs g++ and the ROCm headers")
def test_launch_geometry(tmp_path):
    exe = str(tmp_path / "geometry_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE, "-Wno-attributes",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all"] + SOURCES + ["-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout[-2000:], r.stderr[-4000:])
