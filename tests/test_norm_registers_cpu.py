"""What the compiler keeps in registers of the norm's kernels: few bytes on the stack."""
import os
import re
import shutil
import subprocess

import pytest

from top_sparse_attention_chunked_gb300 import build_lib


def test_rows_stay_in_registers(tmp_path):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("needs nvcc")
    src = os.path.join(build_lib.CSRC, "add_rmsnorm.cu")
    r = subprocess.run([build_lib.nvcc_path(), *build_lib.ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas=-v", "-I",
                        os.path.join(build_lib.HERE, "..", "include"), "-c", src, "-o", str(tmp_path / "norm.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = re.findall(r"add_rmsnorm_kernelILb([01])ELb([01])ELi(\d+)ELi(\d+)E.*?(\d+) bytes spill stores.*?Used (\d+) registers", r.stderr, re.S)
    assert len(kernels) == 16
    for f32, vec, steps, threads, spilled, regs in kernels:
        name = f"FP32 {f32}, vectors {vec}, {steps} steps, {threads} threads"
        assert int(regs) * int(threads) <= 65536, name
        if int(steps) < (4 if vec == "1" else 8) or int(threads) < 1024:
            assert int(spilled) == 0, name                     # 16 elements a thread, or room for 32
        else:
            assert int(spilled) <= 512, f"{name}: {spilled} bytes in {regs} registers"
