"""What the attention side's sources may not hold: its kernels start while their predecessor on the stream still runs
(programmatic dependent launch), and the non-coherent load path is for data that nothing writes while a kernel lives."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "engram_gram_hash_02_gb300", "csrc")


@pytest.mark.parametrize("name", ["heads.cu", "attention.cuh", "attn.cuh", "attn_abi.cu", "attention_bf16.cu", "attention_fp8.cu"])
def test_no_non_coherent_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", code)
