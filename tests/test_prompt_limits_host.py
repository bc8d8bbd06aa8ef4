"""The largest prompts and shared batches that the C ABI takes: rows of a key head are counted in 32 bits, a pair of tiles from any of
them on too. Refused before any CUDA call, so without a GPU."""
import ctypes as C

import pytest

from tests.test_attention_host import E  # noqa: F401
from tests.test_prompt_attention_host import Abi2

MOST = 2 ** 31 - 256


@pytest.mark.parametrize("T,heads", [(2 ** 31 - 1, 2), (MOST + 1, 2), (MOST // 2 + 1, 4), (2 ** 28, 16)])
def test_rows_past_the_most_are_refused(E, T, heads):
    a = Abi2(E)
    rows = a.heads(heads=heads, ts=64 * heads)
    assert a.prompt(T=T, q=rows, out=rows) == -1
    assert "2^31" in a.L.engram_last_error().decode()
    assert a.L.engram_prompt_workspace_bytes(C.byref(a.cache()), heads, T, 1) == 0
    if T < 2 ** 31 and heads == 2:
        batch = a.seqs(batch=T)
        assert a.shared(seqs=batch, q=rows, out=rows) == -1 and "2^31" in a.L.engram_last_error().decode()
        assert a.L.engram_shared_workspace_bytes(C.byref(a.cache()), heads, T, 1) == 0


@pytest.mark.parametrize("T,heads", [(MOST, 2), (MOST // 2, 4)])
def test_the_most_rows_are_taken(E, T, heads):
    """(their workspace is asked for, and one that is too small is what is refused)"""
    a = Abi2(E)
    rows = a.heads(heads=heads, ts=64 * heads)
    need = a.L.engram_prompt_workspace_bytes(C.byref(a.cache()), heads, T, 1)
    assert need > 2 ** 28
    assert a.prompt(T=T, q=rows, out=rows, n=need - 256) == -1
    assert "workspace" in a.L.engram_last_error().decode()
