"""The rings and barriers of the cached attention's kernel for many rows, as a
model on the host (cache_ring_check.cpp) over the stretches of tiles that
fa_cache_geom.h gives each CTA."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "unet_fa_fwd_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path_factory.mktemp("rings") / "cache_ring_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), os.path.join(HERE, "cache_ring_check.cpp")],
                   check=True)
    return lambda arg: subprocess.run([str(exe), arg], capture_output=True, text=True, timeout=300).stdout.strip()


def test_every_use_sees_its_own_tile(model):
    assert model("kernel") == "ok"


def test_the_model_sees_scales_that_are_read_too_early(model):
    assert model("planted") == "stale"
