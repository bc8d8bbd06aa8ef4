"""The prompt kernel's way out, without a GPU: the phases of the barriers that boxes arrive on (csrc/ring.h), compiled as a host
program, and that a block whose waits have run past their limit waits for the boxes that its warps requested last before it leaves
shared memory behind."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "engram_gram_hash_02_gb300", "csrc")


def test_last_requests_of_a_ring(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "ring_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "ring_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


def test_requested_boxes_land_before_a_block_leaves():
    with open(os.path.join(CSRC, "prompt.cuh")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    kernel = code[code.index("prompt_kernel("):]
    end = kernel.index("__syncthreads();", kernel.index("tma_load_4d("))
    roles = kernel[:end]
    assert "drain<kFp8>(" in kernel[end:kernel.index("tcgen05.dealloc")]
    leaving = code[code.index("void drain("):code.index("prompt_kernel(")]
    for request, said, bars in (("tma_load_4d(", "ctl->asked[", ("kFp8 ? &ctl->st_full", "&ctl->full")), ("tma_load_3d(", "ctl->asked_q", ("&ctl->q_full",))):
        assert said in roles[roles.rindex(request) - 600:] and said in leaving, request
        assert all(f"wait_inline(smem_u32({b}" in leaving or f": {b}" in leaving for b in bars), request


@pytest.mark.parametrize("name", ["prompt.cu", "prompt.cuh", "prompt_bf16.cu", "prompt_fp8.cu", "attention_form_bf16.cu", "attention_form_fp8.cu"])
def test_no_non_coherent_loads(name):
    """Kernels start while their predecessor on the stream still runs; that load path is for data that nothing writes meanwhile."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", code)
