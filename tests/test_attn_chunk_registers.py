"""The attention of several new tokens moves registers between its warps: what a role needs has to fit its share.  A form
whose MMA warp kept descriptors on a stack faulted, so no instance has a stack frame or spills."""
import os
import re
import subprocess

import pytest

from w8a8_precision_gemm_gb300 import _build


def resources(report):
    """(kernel, bytes of stack, of spill stores, of spill loads, registers) of each kernel in the assembler's report."""
    found = re.findall(r"entry function '(\w+)'.*?(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads.*?"
                       r"Used (\d+) registers", report, re.S)
    return [(name, *map(int, rest)) for name, *rest in found]


def test_report_is_read():
    text = ("ptxas info    : Compiling entry function 'a1' for 'sm_103a'\nptxas info    : Function properties for a1\n"
            "    16 bytes stack frame, 4 bytes spill stores, 8 bytes spill loads\nptxas info    : Used 40 registers\n")
    assert resources(text) == [("a1", 16, 4, 8, 40)]


def test_no_instance_has_a_stack(tmp_path):
    try:
        cc = _build.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    r = subprocess.run([cc] + _build.FLAGS + ["-Xptxas", "-v", "-c", os.path.join(_build.CSRC, "attn_chunk.cu"), "-o",
                                             str(tmp_path / "attn_chunk.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = [k for k in resources(r.stdout + r.stderr) if "kv_attn_chunk_kernel" in k[0]]
    assert len(kernels) == 4
    for name, stack, stores, loads, registers in kernels:
        assert (stack, stores, loads) == (0, 0, 0), name
        assert registers == 128, name  # at launch: 512 threads share the SM's 65536, and setmaxnreg moves what they have
