"""What the compiler gives the append's kernels (no GPU)."""
import re
import subprocess

from w4_grouped_gemm_gb300 import build


def test_16_bit_append_keeps_its_places(tmp_path):
    """The 16-bit append by runs keeps 64 to 80 registers a thread with one and two heads a thread, and 104 with four,
    so that three or four, and two, of its blocks of 256 fit on an SM.  (With the 8-bit append's code in one template
    and a bound of one block it took 108 to 145, and 8192 tokens of 20 heads of 256 39.5 us in place of 32.9.)"""
    cmd = [build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I", str(build.INCLUDE), "-Xptxas", "-v", "-c",
           str(build.CSRC / "attn_rope.cu"), "-o", str(tmp_path / "x.o")]
    said = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    most = {1: 80, 2: 85, 4: 128}
    seen = 0
    for name, registers in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", said, re.S):
        kernel = re.search(r"rope_append_runs_kernelILb0ELi[01]ELb[01]ELi([124])E", name)
        if kernel:
            seen += 1
            assert int(registers) <= most[int(kernel[1])], name
    assert seen == 12
