"""Refusals of the attention side's binding: an argument that is no tensor is named, whatever it is."""
import pytest
import torch


@pytest.fixture(scope="module")
def E():
    from engram_gram_hash_02_gb300 import build as B
    B.build()
    import engram_gram_hash_02_gb300 as E
    return E


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("v", [None, 3, [1.0]])
def test_a_cache_needs_values(E, v):
    with pytest.raises(TypeError, match="v must be a torch.Tensor"):
        E.KVCache(z(2, 2, 8, 64), v)


@pytest.mark.parametrize("lse", [1, 0, 1.0])
def test_a_number_is_no_log_sum_exp(E, lse):
    cache = E.KVCache.allocate(10, 16, 2, 64, device="cpu")
    with pytest.raises(TypeError, match="lse"):
        E.engram_paged_attention(cache, z(3, 4, 64), z(3, 4, dtype=torch.int32), z(3, dtype=torch.int32), lse=lse)
