"""Set-up once a device (csrc/device_once.h), compiled for the host with g++: each device of a process gets its own, a
failure is tried again, and one kernel's is not another's."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "bitwise_deterministic_shard_gb300", "csrc")


def test_each_device_is_set_up_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "drv")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, os.path.join(HERE, "device_once_driver.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out == ["failed 3 7", "0 1", "1 1", "3 2", "63 1", "64 2", "69 1", "other 1"]


def test_no_limit_is_set_once_a_process():
    """The training kernels' limits of dynamic shared memory go through it."""
    for name in ("attn_train_fwd.cuh", "attn_train_bwd.cuh", "norm_kernels.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "cudaFuncSetAttribute" not in text, name
        assert re.search(r"allow_smem\(|TileSmem", text), name
