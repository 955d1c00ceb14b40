"""What the entry points leave behind when a CUDA call fails, on the CPU: their host code against a runtime made for it."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gradient_quantization_communication_b200", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_a_failed_call_leaves_no_error_for_the_next_launch(tmp_path):
    exe = str(tmp_path / "cuda_error_check")
    sources = [os.path.join(CSRC, "gq_adamw_api.cu"), os.path.join(CSRC, "gq_api.cu"),
               os.path.join(ROOT, "tests", "cuda_error_check.cpp")]
    # entry points that the check does not call, and the kernels behind them, are dropped by the linker
    subprocess.run(["g++", "-O1", "-std=c++17", "-ffunction-sections", "-Wl,--gc-sections", "-I" + os.path.join(ROOT, "include"),
                    "-I" + CSRC, "-I" + os.path.join(CUDA, "include"), "-x", "c++", *sources, "-o", exe, "-ldl"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
