"""The example that serves a layer (Engram residual, prompt, paged cache, decode steps): decoding token by token
gives the logits that the same tokens give as prompts."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_decoded_logits_equal_prompted_logits(fmt):
    spec = importlib.util.spec_from_file_location("decode_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, same = m.main(["--cache", fmt, "--steps", "24"])
    # the two ways differ by the summation order of plain fp32 products (about 1e-6 of a row's size); a cached
    # value that then rounds to its neighbour moves by 2^-8 (bf16) or 2^-4 (FP8) in one of thousands: of the
    # bf16 output's own step, 2^-8, at most
    assert same and off <= 2.0 ** -8
