"""The weight gradient's ring of stages (gq_ring.cuh, plain C++) compiled for the CPU and run under a model of the
barriers with random delays: no wait may pass before the phase that it means is complete.  No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_check")
    inc = os.path.join(ROOT, "gradient_quantization_communication_b200", "csrc")
    src = os.path.join(ROOT, "tests", "ring_check.cpp")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I" + inc, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_no_wait_passes_early(exe, seed):
    r = subprocess.run([exe, str(seed), "400"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert "early in 0, stuck 0" in r.stdout


def test_the_model_finds_a_skipped_phase(exe):
    """One "full" barrier a stage, waited for at every second use only, passes early; the model has to see it."""
    r = subprocess.run([exe, "1", "400", "plain"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 1 and "early in 0" not in r.stdout, r.stdout
