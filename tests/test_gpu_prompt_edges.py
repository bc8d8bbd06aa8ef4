"""Prompts at the edges of their range: tokens that see nothing beside values that are not finite, masks of the type's extremes,
scores that rise far within a tile of keys, a cap far below the scale, and workspaces whose start is not zero."""
import numpy as np
import pytest
import torch

from tests import _attention as H
from tests import _prompts as P
from tests.test_gpu_prompt_attention import ZERO, cu_of, randn, word

pytestmark = pytest.mark.gpu
DEV = "cuda"


def spoil(cache, table, b, j, at):
    """A value that is not finite at position `at` of key j of sequence b, in every head: NaN, and over bf16 an infinity next to it."""
    s = H.slots_of(table, b, j, j + 1, cache.page_size)[0]
    cache.v[s // cache.page_size, :, s % cache.page_size, at] = float("nan") if cache.fmt == "bf16" else 0x7F
    if cache.fmt == "bf16":
        cache.v[s // cache.page_size, :, s % cache.page_size, at + 1] = float("inf")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 6), (256, 16)])
@pytest.mark.parametrize("new,old", [([70], [2930]), ([64] * 100, [300] * 100)])   # few pairs, cut many times; many pairs, some of them whole
def test_a_token_that_sees_nothing_gives_zeros_beside_values_that_are_not_finite(new, old, D, page, fmt):
    E = H.pkg()
    lens = [n + m for n, m in zip(new, old)]
    cache, table = H.filled(lens, page, 4, D, fmt, 60)
    T = sum(new)
    q = randn(61, (T, 8, D))
    doc = np.zeros(T, np.int32)
    empty = np.arange(T) % 7 == 3
    doc[empty] = 10 ** 6
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    want, want_lse = E.engram_prompt_attention(cache, q, *args, doc_starts=P.dev(doc), lse=True)
    P.check_prompt(cache, table, new, lens, q, want, want_lse, D ** -0.5, doc_starts=doc)
    at = D - 5
    for b in range(len(lens)):
        spoil(cache, table, b, 10, at)                       # every token that sees anything sees it
    out, lse = (torch.full_like(x, 7.0) for x in (want, want_lse))
    E.engram_prompt_attention(cache, q, *args, doc_starts=P.dev(doc), out=out, lse=lse)
    e = torch.from_numpy(empty).to(DEV)
    assert not out[e].any() and bool(torch.isneginf(lse[e]).all())
    hit = [at, at + 1] if fmt == "bf16" else [at]
    rest = [d for d in range(D) if d not in hit]
    assert not torch.isfinite(out[~e][..., hit]).any()
    assert torch.equal(out[~e][..., rest], want[~e][..., rest]) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("D", [64, 256])
def test_scores_that_are_all_minus_infinity_give_zeros_whatever_the_values(D):
    E, new, lens = H.pkg(), [200], [200]
    cache, table = H.filled(lens, 16, 1, D, "bf16", 62)
    q = randn(63, (200, 4, D))
    q[..., 0] = 1.0
    for s in H.slots_of(table, 0, 0, 200, 16):
        cache.k[s // 16, 0, s % 16, 0] = float("-inf")
    spoil(cache, table, 0, 3, 5)
    spoil(cache, table, 0, 150, D - 2)
    out, lse = E.engram_prompt_attention(cache, q, P.dev([0, 200]), P.dev(table), P.dev(lens), causal=False, lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("fmt,D,slopes", [("bf16", 64, False), ("bf16", 256, False), ("fp8", 128, True)])
def test_masks_of_the_types_extremes(fmt, D, slopes):
    """Documents that start at the largest and the smallest number there is, and prefixes that end there."""
    E, new, lens = H.pkg(), [200, 130, 300], [500, 130, 300]
    cache, table = H.filled(lens, 16, 2, D, fmt, 64)
    T = sum(new)
    q = randn(65, (T, 8, D))
    top, low = 2 ** 31 - 1, -2 ** 31
    doc, ends = np.zeros(T, np.int32), np.zeros(T, np.int32)
    for i, x in enumerate((top, low, top - 126, top - 127, 2 ** 31 - 256, 100)):
        doc[5 + 3 * i::40] = x
    ends[200:330:9] = top
    ends[203:330:9] = low
    sl = P.alibi(8) if slopes else None
    out, lse = torch.full_like(q, 7.0), torch.full((T, 8), 7.0, device=DEV)
    E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), doc_starts=P.dev(doc), prefix_ends=P.dev(ends),
                              slopes=None if sl is None else P.dev(sl, torch.float32), out=out, lse=lse)
    assert not out[5::40].any() and bool(torch.isneginf(lse[5::40]).all())
    P.check_prompt(cache, table, new, lens, q, out, lse, D ** -0.5, doc_starts=doc, prefix_ends=ends, slopes=sl)
