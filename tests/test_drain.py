"""Copies in flight when a bounded wait runs out: the kernels' counting against a model of their barriers, on
the host (no wait is made to run out on a GPU with copies in flight)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "hadamard_bit_quant_hbl_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    exe = str(tmp_path_factory.mktemp("drain") / "model")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "drain_model.cpp"), "-o", exe], check=True)
    return exe


def test_drain_waits_for_every_copy_in_flight(model):
    res = subprocess.run([model], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout
