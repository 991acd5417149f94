"""Index arithmetic of the matrix products, compiled for the host and walked over sizes on the CPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_index_arithmetic_stays_in_range(tmp_path):
    exe = str(tmp_path / "gemm_index")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "combine_moe_layout_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "gemm_index.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
