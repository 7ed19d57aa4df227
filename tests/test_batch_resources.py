"""ptxas report of the batched attention (on the CPU): both head sizes must
compile without spills at the register split that the kernel launches with."""
import os
import re
import shutil
import subprocess

import pytest

from chunk_causal_attention_block_b200 import build as wfbuild


def test_batched_attention_compiles_without_spills(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = os.path.join(wfbuild.CSRC, "batch_attn.cu")
    r = subprocess.run([nvcc] + wfbuild.NVCC_FLAGS + ["-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "a.o")],
                       capture_output=True, text=True, check=True)
    report = r.stdout + r.stderr
    blocks = re.findall(r"Compiling entry function '([^']*)'.*?\n(.*?)\nptxas info\s+: Used (\d+) registers", report,
                        flags=re.S)
    assert len([b for b in blocks if "batch_attn_kernel" in b[0]]) == 2, report
    for name, props, regs in blocks:
        assert "0 bytes spill stores, 0 bytes spill loads" in props, (name, props)
        assert int(regs) <= 168, (name, regs)
