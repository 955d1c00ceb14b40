"""The 8-bit products' places in shared memory, on the CPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_stages_and_parts_are_aligned_wherever_shared_memory_begins(tmp_path):
    exe = str(tmp_path / "fp8_shared_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "gradient_quantization_communication_b200", "csrc"),
                    os.path.join(ROOT, "tests", "fp8_shared_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
