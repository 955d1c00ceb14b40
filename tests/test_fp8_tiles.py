"""The 8-bit products' schedules, walked over on the CPU: every stage of every tile once, for many sizes."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_stage_is_taken_once(tmp_path):
    exe = str(tmp_path / "fp8_tiles_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "gradient_quantization_communication_b200", "csrc"),
                    os.path.join(ROOT, "tests", "fp8_tiles_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
