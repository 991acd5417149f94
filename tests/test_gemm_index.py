"""Index arithmetic of the matrix products, compiled for the host and walked over sizes on the CPU; what
their inline assembly declares; how the resource table names them."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_index_arithmetic_stays_in_range(tmp_path):
    exe = str(tmp_path / "gemm_index")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "combine_moe_layout_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "gemm_index.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_inline_assembly_names_the_m0_it_writes():
    """The compiler keeps values of its own in m0: a statement that writes it says so."""
    csrc = os.path.join(ROOT, "combine_moe_layout_amd", "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        for text in re.findall(r"asm volatile\((.*?)\);", open(os.path.join(csrc, name)).read(), re.S):
            if re.search(r"\bs_\w+ m0,", text):
                seen += 1
                assert re.search(r':\s*"m0"\s*$', text), (name, text)
    assert seen >= 3


def test_resource_table_names_kernels():
    from combine_moe_layout_amd.build import kernel_label
    assert kernel_label("void ep::(anonymous namespace)::gemm_few_kernel<0, false, true, 2, 1>(ep::GemmArgs)") == \
        "gemm_few_kernel<0, false, true, 2, 1>"
    assert kernel_label("ep::layout_count_kernel(long const*, int)") == "layout_count_kernel"
