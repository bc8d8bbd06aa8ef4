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


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D,form", [(64, False), (64, True), (192, False)])
def test_scores_that_rise_by_thirty_within_a_tile_of_keys(fmt, D, form):
    """Three keys of 256 count: one of the second tile of keys, which is taken first, with score 0, and two of the first tile, of 20.1
    (29 to 29.2 in units of log 2, below what moves the maximum) and 21.4 (30.9 to 31.1). Their weights are rounded once: by 2^-8
    of themselves. The first one's value alone is not zero; its 64 different multiples of the weight tell how far the weight is off."""
    E, B, n, Hk, G = H.pkg(), 20, 8, 8, 32
    page, lens = 16, [256] * B
    cache, table = H.filled(lens, page, Hk, D, fmt, 66)
    k, v = (torch.zeros((256, Hk, D), device=DEV) for _ in range(2))
    k[:, :, 4] = -1.0                                        # the others: -200
    for j, row in ((131, (0, 0, 0, 0, 0)), (5, (20, 0.125, 0, 1, 0)), (70, (20, 1.375, 0.0625, 1, 0))):
        k[j, :, :5] = torch.tensor(row, dtype=torch.float32, device=DEV)
    v[5, :, :64] = 1 + torch.arange(64, device=DEV) / 64.0
    if fmt == "fp8":
        v[5, :, :64] = (1 + torch.arange(64, device=DEV) % 8 / 8.0) * 2.0 ** (torch.arange(64, device=DEV) // 8 % 4)
    for b in range(B):
        E.engram_kv_write(cache, k, v, torch.from_numpy(H.slots_of(table, b, 0, 256, page)).to(DEV))
    q = torch.zeros((B * n, Hk * G, D), dtype=torch.bfloat16, device=DEV)
    q[..., :3], q[..., 4] = 1.0, 200.0
    q[..., 3] = (torch.rand((B * n, Hk * G), generator=torch.Generator(device=DEV).manual_seed(67), device=DEV) * 0.075 - 0.015).bfloat16()
    how = dict(slopes=torch.zeros(Hk * G, device=DEV)) if form else {}
    out = E.engram_prompt_attention(cache, q, P.dev(np.arange(B + 1) * n), P.dev(table), P.dev(lens), scale=1.0, **how)
    free = q[..., 3].double()
    s0, s1, s2 = torch.zeros_like(free), 20.125 + free, 21.4375 + free
    weight = torch.exp(s1) / (torch.exp(s0) + torch.exp(s1) + torch.exp(s2))
    want = weight[..., None] * v[5, 0].double()
    got = out.double()
    half_step = torch.exp2(torch.floor(torch.log2(got.abs().clamp_min(2.0 ** -100))) - 8)
    # the weight's one rounding, the output's, and 2^-16 for scores of 21 and sums in 32 bits
    bound = half_step + (2.0 ** -8 + 2.0 ** -16) * want
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / want.clamp_min(1e-30)).max() * 256)


@pytest.mark.parametrize("rise", [31.0, 100.0, 200.0, 1e6])
def test_scores_that_rise_by_any_number(rise):
    """Every key half a tile on, in the order in which they are taken, has a score `rise` larger: its value is what comes out."""
    E, lens = H.pkg(), [1024]
    cache, table = H.filled(lens, 16, 1, 64, "bf16", 72)
    slots = torch.from_numpy(H.slots_of(table, 0, 0, 1024, 16)).to(DEV)
    step = np.concatenate([[2 * (7 - j // 128) + (j % 128) // 64] for j in range(1024)])
    k, v = (torch.zeros((1024, 1, 64), device=DEV) for _ in range(2))
    k[:, 0, 0] = torch.as_tensor(step - 7.0, device=DEV)
    v[:] = torch.as_tensor(1.0 + step, device=DEV)[:, None, None]
    E.engram_kv_write(cache, k, v, slots)
    q = torch.zeros((130, 2, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    for cap, slopes in ((0.0, None), (1e16, None), (0.0, torch.zeros(2, device=DEV))):
        out, lse = E.engram_prompt_attention(cache, q, P.dev([0, 130]), P.dev(table), P.dev(lens), scale=rise, causal=False, cap=cap,
                                             slopes=slopes, lse=True)
        assert bool((out == 16.0).all())
        # 64 keys of the largest score: fp32 of it, and of the logarithm (a capped one: 2^-19 of itself)
        top = cap * np.tanh(8 * rise / cap) if cap else 8 * rise
        assert float((lse.double() - (top + np.log(64.0))).abs().max()) <= top * (2.0 ** -21 + (2.0 ** -19 if cap else 0)) + 2.0 ** -20


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_scores_at_the_end_of_their_range(fmt):
    """Scores of almost 2^26 of either sign: a row's weights share a factor of up to 2^4, and values of 2^80 stay in range."""
    E, lens = H.pkg(), [600]
    cache, table = H.filled(lens, 16, 1, 64, fmt, 74)
    slots = torch.from_numpy(H.slots_of(table, 0, 0, 600, 16)).to(DEV)
    k, v = (torch.zeros((600, 1, 64), device=DEV) for _ in range(2))
    k[:, 0, 0] = 2.0 + torch.arange(600, device=DEV) % 14
    v[:] = (1.0 + torch.arange(600, device=DEV) % 14)[:, None, None] * 2.0 ** 80
    E.engram_kv_write(cache, k, v, slots)
    rng = np.random.default_rng(75)
    q = torch.zeros((400, 2, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = torch.from_numpy(rng.uniform(1, 4.3e6, (400, 2)) * rng.choice([-1, 1], (400, 2))).to(DEV)
    out = E.engram_prompt_attention(cache, q, P.dev([0, 400]), P.dev(table), P.dev(lens), scale=1.0, causal=False)
    want = torch.where(q[..., :1] > 0, 14.0, 1.0).double() * 2.0 ** 80
    far = q[..., :1].abs() > 100.0                           # the next key's score is that far below: its weight is nothing
    assert bool(far.float().mean() > 0.99)
    assert bool(((out.double() - want).abs() <= 2.0 ** -7 * want)[far.expand_as(out)].all())   # the weight's rounding, and the output's


@pytest.mark.parametrize("new,old", [([64] * 100, [300] * 100), ([70], [2930])])
def test_prompts_do_not_depend_on_the_workspaces_start(new, old):
    """The zeroed start belongs to the one-token calls: prompts neither read nor write it, so that a call that gave up (a wait past
    its limit) leaves nothing behind for the next one. What else a workspace holds does not count either."""
    E = H.pkg()
    lens = [n + m for n, m in zip(new, old)]
    cache, table = H.filled(lens, 16, 4, 128, "bf16", 70)
    T = sum(new)
    q = randn(71, (T, 8, 128))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    want, want_lse = E.engram_prompt_attention(cache, q, *args, lse=True)
    P.check_prompt(cache, table, new, lens, q, want, want_lse, 128 ** -0.5)
    for byte in (0x01, 0xA5, 0xFF):
        ws = torch.full((E.prompt_workspace_bytes(cache, 8, T, len(new)),), byte, dtype=torch.uint8, device=DEV)
        out, lse = torch.full_like(q, float("nan")), torch.full_like(want_lse, float("nan"))
        for _ in range(2):
            E.engram_prompt_attention(cache, q, *args, out=out, lse=lse, workspace=ws)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert bool((ws[:ZERO] == byte).all())


@pytest.mark.parametrize("slopes", [False, True])
def test_a_cap_far_below_the_scale(slopes):
    """scale / cap is past what 32 bits hold: every score is 0 or +-cap, which is next to nothing, and all weights are equal."""
    E, new, lens = H.pkg(), [60, 7], [60, 300]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 68)
    q = randn(69, (67, 4, 64))
    q[::3] = 0.0
    out, lse = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), scale=2.0 ** 70, cap=2.0 ** -60, causal=False,
                                         slopes=torch.zeros(4, device=DEV) if slopes else None, lse=True)
    P.check_prompt(cache, table, new, lens, torch.zeros_like(q), out, lse, 1.0, causal=False)


@pytest.mark.parametrize("fmt,D", [("bf16", 240), ("fp8", 256), ("bf16", 64), ("fp8", 128)])
def test_rows_one_by_one_in_short_pieces_many_times(fmt, D):
    """Pages that do not divide into boxes, key tiles in ones and twos: no wait is left behind, and every call gives the same bits."""
    E = H.pkg()
    new = [2, 27, 1, 1, 0, 44, 23, 32, 0, 2, 0, 35, 11, 2, 33, 1]
    lens = [n + m for n, m in zip(new, [27, 388, 141, 372, 278, 152, 140, 378, 383, 111, 0, 2, 385, 187, 22, 184])]
    cache, table = H.filled(lens, 7, 3, D, fmt, 76, "padded")
    T = sum(new)
    q = randn(77, (T, 48, D))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    err = word()
    ws = E.prompt_workspace(cache, 48, T, len(new))
    out, lse = E.engram_prompt_attention(cache, q, *args, lse=True, workspace=ws, err=err)
    P.check_prompt(cache, table, new, lens, q, out, lse, D ** -0.5)
    again, again_lse = torch.empty_like(out), torch.empty_like(lse)
    plan = E.PromptAttentionPlan(cache, q, *args, out=again, lse=again_lse, workspace=ws, err=err)
    for _ in range(2000):
        plan.run()
    assert int(err) == 0 and torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("fmt,page", [("bf16", 16), ("fp8", 16), ("bf16", 5)])
def test_two_tiles_with_long_joins_before_one_tile_many_times(fmt, page):
    """Long sequences of two tiles, cut many times and joined by one block's warps, each followed by ones of a single tile."""
    E = H.pkg()
    new, old = [64, 9, 70, 5] * 10, [6000, 900, 2500, 1300] * 10
    lens = [n + m for n, m in zip(new, old)]
    cache, table = H.filled(lens, page, 4, 64, fmt, 78)
    T = sum(new)
    q = randn(79, (T, 16, 64))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    err = word()
    out, lse = E.engram_prompt_attention(cache, q, *args, lse=True, err=err)
    P.check_prompt(cache, table, new, lens, q, out, lse, 0.125, rows=np.arange(0, T, 13))
    again, again_lse = torch.empty_like(out), torch.empty_like(lse)
    plan = E.PromptAttentionPlan(cache, q, *args, out=again, lse=again_lse, err=err)
    for _ in range(500):
        plan.run()
    assert int(err) == 0 and torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("Hq", [8, 6])                       # queries as boxes, and row by row
def test_outputs_in_the_place_of_queries(Hq):
    """Whole pairs, cut ones and rows that see nothing; a batch that shares a prefix."""
    E, new, lens = H.pkg(), [700, 3, 90, 20], [700, 4000, 5000, 10]
    cache, table = H.filled(lens, 16, 2, 128, "bf16", 80)
    T = sum(new)
    q = randn(81, (T, Hq, 128))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    want = E.engram_prompt_attention(cache, q, *args)
    same = q.clone()
    assert E.engram_prompt_attention(cache, same, *args, out=same) is same and torch.equal(same, want)
    q = randn(82, (3, Hq, 128))
    args = P.dev(table[2:3]), P.dev([5000]), P.dev([0, 3]), P.dev(table[[0, 1, 3]]), P.dev([700, 0, 10])
    want = E.engram_shared_attention(cache, q, *args)
    same = q.clone()
    assert E.engram_shared_attention(cache, same, *args, out=same) is same and torch.equal(same, want)


def test_views_that_repeat_rows():
    """Strides of zero, which no tensor map takes: one query row for all heads, one key head's rows for all."""
    E, new, lens = H.pkg(), [150, 40], [300, 40]
    cache, table = H.filled(lens, 16, 1, 64, "bf16", 83)
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    q = randn(84, (190, 1, 64)).expand(190, 8, 64)
    wide = E.KVCache(cache.k.expand(-1, 4, -1, -1), cache.v.expand(-1, 4, -1, -1))
    full = E.KVCache(wide.k.contiguous(), wide.v.contiguous())
    want, want_lse = E.engram_prompt_attention(full, q.contiguous(), *args, lse=True)
    P.check_prompt(full, table, new, lens, q, want, want_lse, 0.125)
    for c, x in ((wide, q), (wide, q.contiguous()), (full, q)):
        out, lse = E.engram_prompt_attention(c, x, *args, lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
