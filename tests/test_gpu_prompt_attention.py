"""Attention of all tokens of prompts through the C ABI against the 64-bit oracle: masks, score forms, cache formats and
layouts, ragged batches, and everything that a token may not see. Bounds come from the formulas' roundings."""
import numpy as np
import pytest
import torch

from tests import _attention as H
from tests import _prompts as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
ZERO = 16384


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def randn(seed, shape, std=1.0, dtype=torch.bfloat16):
    return (std * torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)).to(dtype)


def cu_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def documents(new, lens, length, seed):
    """First positions of documents of about `length` tokens, per new token."""
    rng = np.random.default_rng(seed)
    got = []
    for n, m in zip(new, lens):
        starts = np.unique(np.concatenate([[0], rng.integers(0, max(m, 1), size=m // length + 1)]))
        p = m - n + np.arange(n)
        got.append(starts[np.maximum(np.searchsorted(starts, p, side="right") - 1, 0)])
    return np.concatenate(got).astype(np.int32)


def prefixes(new, lens, seed):
    """A third of each prompt's new tokens is seen both ways."""
    return np.concatenate([np.full(n, m - n + n // 3) for n, m in zip(new, lens)]).astype(np.int32)


CASES = [
    # new tokens, tokens cached before, page, Hq, Hk, D, cache, layout, mask, cap, slopes
    ([1], [0], 16, 8, 2, 64, "bf16", "hnd", "causal", 0.0, False),
    ([37], [0], 16, 32, 8, 128, "bf16", "hnd", "causal", 0.0, False),
    ([300], [0], 64, 4, 1, 128, "bf16", "nhd", "causal", 0.0, False),
    ([129, 1, 0, 64], [0, 700, 31, 5], 24, 6, 2, 96, "bf16", "padded", "causal", 0.0, False),
    ([700], [0], 1, 2, 2, 64, "bf16", "hnd", "causal", 0.0, False),
    ([257, 255], [511, 1], 7, 3, 3, 256, "bf16", "nhd", "causal", 0.0, False),
    ([5] * 6, [3, 400, 1000, 0, 129, 77], 64, 32, 8, 128, "bf16", "hnd", "causal", 0.0, False),
    ([5] * 6, [3, 400, 1000, 0, 129, 77], 16, 16, 1, 128, "fp8", "nhd", "causal", 0.0, True),
    ([600], [0], 32, 8, 2, 192, "fp8", "padded", "causal", 30.0, False),
    ([530, 40], [100, 900], 16, 4, 4, 32, "fp8", "hnd", "docs", 0.0, False),
    ([1111], [0], 32, 4, 2, 256, "bf16", "hnd", "docs", 50.0, False),
    ([400, 333], [0, 1700], 64, 8, 8, 64, "bf16", "hnd", "window", 0.0, True),
    ([400, 333], [0, 1700], 64, 8, 2, 128, "fp8", "hnd", "window", 0.0, False),
    ([211, 500], [0, 64], 24, 12, 12, 64, "bf16", "hnd", "prefix", 0.0, True),
    ([211, 500], [0, 64], 24, 5, 1, 80, "bf16", "nhd", "prefix", 20.0, True),
    ([70, 300], [900, 0], 16, 4, 1, 128, "bf16", "hnd", "full", 0.0, False),
    ([70, 300], [900, 0], 16, 4, 1, 128, "fp8", "hnd", "full", 5.0, True),
    ([65, 130], [10, 20], 128, 34, 2, 48, "bf16", "hnd", "causal", 0.0, False),
    ([3, 2], [50, 8], 16, 256, 1, 16, "bf16", "hnd", "causal", 0.0, False),
    ([400], [0], 16, 4, 2, 64, "bf16", "hnd", "docs+window", 0.0, False),
    ([400], [100], 16, 4, 2, 64, "bf16", "hnd", "prefix+window", 0.0, False),
    ([400], [100], 16, 4, 2, 160, "fp8", "hnd", "prefix+docs", 0.0, False),
]


def masks(mask, new, lens, seed):
    how = {}
    if "docs" in mask:
        how["doc_starts"] = documents(new, lens, 90, seed)
    if "prefix" in mask:
        how["prefix_ends"] = prefixes(new, lens, seed)
    if "window" in mask:
        how["window"] = 150
    return how | {"causal": mask != "full"}


@pytest.mark.parametrize("new,old,page,Hq,Hk,D,fmt,layout,mask,cap,slopes", CASES)
def test_prompts_match_the_formula(new, old, page, Hq, Hk, D, fmt, layout, mask, cap, slopes):
    E, seed = H.pkg(), sum(new) + D
    lens = [n + m for n, m in zip(new, old)]
    cache, table = H.filled(lens, page, Hk, D, fmt, seed, layout, spread=1.0)
    T = sum(new)
    q = randn(seed, (T, Hq, D), cap / 4 if cap else 1.5)
    sl = P.alibi(Hq) if slopes else None
    how = masks(mask, new, lens, seed)
    err = word()
    out, lse = torch.full_like(q, float("nan")), torch.full((T, Hq), float("nan"), device=DEV)
    ws = E.prompt_workspace(cache, Hq, T, len(new))
    E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), cap=cap, slopes=None if sl is None else P.dev(sl, torch.float32),
                              out=out, lse=lse, workspace=ws, err=err,
                              **{k: P.dev(x) if isinstance(x, np.ndarray) else x for k, x in how.items()})
    assert int(err) == 0 and not ws[:ZERO].any()
    P.check_prompt(cache, table, new, lens, q, out, lse, D ** -0.5, cap=cap, slopes=sl, **how)


def test_strided_rows_and_a_scale_of_their_own():
    """Queries packed with keys and values in one row, outputs heads-first; a scale that is not the default."""
    E, new, lens = H.pkg(), [200, 33], [200, 90]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 5)
    rows = randn(6, (233, 10, 64))
    q = rows[:, 1:7]
    out = torch.full((6, 240, 64), float("nan"), dtype=torch.bfloat16, device=DEV).transpose(0, 1)[3:236]
    lse = torch.empty((233, 6), device=DEV)
    got = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), scale=0.3, out=out, lse=lse)
    assert got[0] is out
    P.check_prompt(cache, table, new, lens, q, out, lse, 0.3)


def test_rows_of_no_sequence_are_left_as_they_were():
    E, new, lens = H.pkg(), [20, 0, 140], [50, 0, 140]
    cache, table = H.filled(lens, 16, 2, 128, "bf16", 7)
    q = randn(8, (300, 8, 128))
    out, lse = torch.full_like(q, 7.0), torch.full((300, 8), 7.0, device=DEV)
    cu = cu_of(new) + 11
    err = word()
    E.engram_prompt_attention(cache, q, P.dev(cu), P.dev(table), P.dev(lens), out=out, lse=lse, err=err)
    assert int(err) == 0
    for rows in (slice(0, 11), slice(171, 300)):
        assert bool((out[rows] == 7).all()) and bool((lse[rows] == 7).all())
    P.check_prompt(cache, table, new, lens, q[11:171], out[11:171], lse[11:171], 128 ** -0.5)


def test_no_tokens_no_sequences_and_sequences_without_new_tokens():
    E = H.pkg()
    cache, table = H.filled([40], 16, 2, 64, "bf16", 9)
    none = E.engram_prompt_attention(cache, randn(1, (0, 4, 64)), P.dev([0, 0]), P.dev(table), P.dev([40]))
    assert none.shape == (0, 4, 64)
    q = randn(2, (3, 4, 64))
    out, lse = torch.full_like(q, 3.0), torch.full((3, 4), 3.0, device=DEV)
    E.engram_prompt_attention(cache, q, P.dev([0]), P.dev(table[:0]), P.dev(np.zeros(0)), out=out, lse=lse)
    E.engram_prompt_attention(cache, q, P.dev([0, 0]), P.dev(table), P.dev([40]), out=out, lse=lse)
    assert bool((out == 3).all()) and bool((lse == 3).all())


def test_tokens_that_see_nothing_give_zeros():
    """Documents that start behind a token, a sequence without a cached token, more new tokens than the length counts."""
    E, new, lens = H.pkg(), [200, 30, 50], [200, 0, 20]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 10)
    q = randn(11, (280, 4, 64))
    doc = np.zeros(280, np.int32)
    doc[20:60] = 10 ** 6
    doc[100] = 101
    doc[120:125] = -5
    err = word()
    out, lse = torch.full_like(q, float("nan")), torch.full((280, 4), float("nan"), device=DEV)
    E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), doc_starts=P.dev(doc), out=out, lse=lse, err=err)
    assert int(err) == E.ERR_SEQ_LEN
    assert not out[20:60].any() and not out[100].any() and not out[200:260].any()
    P.check_prompt(cache, table, new, lens, q, out, lse, 64 ** -0.5, doc_starts=doc)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_what_a_token_does_not_see_has_no_part_in_it(fmt):
    """Infinities and NaN in keys and values that some tokens of a tile see and others do not."""
    E, new, lens = H.pkg(), [300, 290], [300, 421]
    cache, table = H.filled(lens, 16, 2, 64, fmt, 12)
    q = randn(13, (590, 8, 64))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    doc = documents(new, lens, 100, 3)
    want = [E.engram_prompt_attention(cache, q, *args, doc_starts=P.dev(doc), lse=True)]
    P.check_prompt(cache, table, new, lens, q, *want[0], 64 ** -0.5, doc_starts=doc)
    bad = {0: [3, 150, 151, 260], 1: [0, 131, 300, 420]}
    kinds = iter([float("inf"), float("nan"), float("-inf"), float("nan")] * 2)
    for b, keys in bad.items():
        for j in keys:
            s = H.slots_of(table, b, j, j + 1, 16)[0]
            x = next(kinds)
            for t, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
                if fmt == "bf16":
                    t[s // 16, :, s % 16, 5::9] = x
                elif x == x:
                    scales[s // 16, :, s % 16, 0] = 255
                else:
                    t[s // 16, :, s % 16, 5::9] = 0x7F
    out, lse = E.engram_prompt_attention(cache, q, *args, doc_starts=P.dev(doc), lse=True)
    clean, t0 = [], 0
    for b, (n, m) in enumerate(zip(new, lens)):
        for i in range(n):
            p = m - n + i
            if not any(doc[t0 + i] <= j <= p for j in bad[b]):
                clean.append(t0 + i)
        t0 += n
    dirty = np.setdiff1d(np.arange(590), clean)
    assert 50 < len(clean) and 50 < len(dirty)
    assert torch.equal(out[clean], want[0][0][clean]) and torch.equal(lse[clean], want[0][1][clean])
    # a token that sees one has it in its result: NaN in a key or a value reaches every head's lse or out
    assert not torch.isfinite(out[dirty]).all(-1).all(-1).any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attended_values_that_are_not_finite_come_out_so(fmt):
    """An infinity or a NaN among the values spoils the positions that it stands in, for the tokens that see it alone."""
    E, new, lens = H.pkg(), [260], [260]
    cache, table = H.filled(lens, 16, 1, 64, fmt, 14)
    q = randn(15, (260, 4, 64))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    want = E.engram_prompt_attention(cache, q, *args)
    s = H.slots_of(table, 0, 200, 201, 16)[0]
    if fmt == "bf16":
        cache.v[s // 16, 0, s % 16, 7] = float("inf")
        hit = [7]
    else:
        cache.v[s // 16, 0, s % 16, 7] = 0x7F
        hit = [7]
    got = E.engram_prompt_attention(cache, q, *args)
    keep = [d for d in range(64) if d not in hit]
    assert torch.equal(got[:200], want[:200])
    assert not torch.isfinite(got[200:, :, hit]).any()
    assert torch.equal(got[200:][..., keep], want[200:][..., keep]) or \
        float((got[200:][..., keep].float() - want[200:][..., keep].float()).abs().max()) <= 2 ** -6


def test_pages_outside_the_cache_hide_their_tokens():
    E, new, lens = H.pkg(), [150, 20], [150, 500]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 16)
    q = randn(17, (170, 4, 64))
    lost = table.copy()
    lost[0, 3], lost[1, 20], lost[1, 21] = -1, cache.num_pages, 2 ** 31 - 1
    err = word()
    out, lse = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(lost), P.dev(lens), lse=True, err=err)
    assert int(err) == E.ERR_PAGE
    P.check_prompt(cache, table, new, lens, q, out, lse, 64 ** -0.5, hidden=[list(range(48, 64)), list(range(320, 352))])


def test_lengths_and_starts_that_do_not_fit_are_clamped_and_reported():
    E, lens = H.pkg(), [64, 64]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 18)
    q = randn(19, (100, 4, 64))
    want = E.engram_prompt_attention(cache, q, P.dev([0, 40, 100]), P.dev(table), P.dev([64, 64]), lse=True)
    for cu, sl in (([0, 40, 100], [64, 1000]), ([-7, 40, 100], [64, 64]), ([0, 40, 2 ** 31 - 1], [64, 64])):
        err = word()
        got = E.engram_prompt_attention(cache, q, P.dev(cu), P.dev(table), P.dev(sl), lse=True, err=err)
        assert int(err) & E.ERR_SEQ_LEN
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for cu, sl in (([50, 20, 20], [64, 64]), ([0, 0, 40], [64, -3])):
        err = word()
        out, lse = torch.full_like(q, 5.0), torch.full((100, 4), 5.0, device=DEV)
        E.engram_prompt_attention(cache, q, P.dev(cu), P.dev(table), P.dev(sl), out=out, lse=lse, err=err)
        assert int(err) & E.ERR_SEQ_LEN
        if cu[0] == 50:
            assert bool((out == 5).all())
        else:
            assert not out[:40].any() and bool((out[40:] == 5).all()) and bool(torch.isneginf(lse[:40]).all())


def test_scores_of_minus_infinity_and_large_ones():
    """Keys whose score is -inf take no weight; scores of 1e4 keep the softmax in range."""
    E, new, lens = H.pkg(), [140], [140]
    cache, table = H.filled(lens, 16, 1, 64, "bf16", 20)
    q = torch.zeros((140, 2, 64), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    slots = H.slots_of(table, 0, 0, 140, 16)
    for j, s in enumerate(slots):
        cache.k[s // 16, 0, s % 16, 0] = float("-inf") if j % 3 == 0 else 100.0 * (j % 7)
    out, lse = E.engram_prompt_attention(cache, q, P.dev([0, 140]), P.dev(table), P.dev(lens), scale=100.0, lse=True)
    assert not out[0].any() and bool(torch.isneginf(lse[0]).all())       # only a key of -inf
    P.check_prompt(cache, table, new, lens, q, out, lse, 100.0, hidden=[list(range(0, 140, 3))])


def test_a_form_without_effect_and_one_token_equal_the_one_token_call():
    """One new token per sequence: engram_prompt_attention is engram_paged_attention, to the weights' rounding."""
    E, lens = H.pkg(), [1, 700, 64, 0, 1300]
    for fmt in ("bf16", "fp8"):
        cache, table = H.filled(lens, 16, 2, 128, fmt, 21)
        q = randn(22, (5, 8, 128))
        for how in (dict(), dict(cap=20.0), dict(slopes=P.dev(P.alibi(8), torch.float32)), dict(window=100)):
            a, la = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), lse=True, **how)
            b, lb = E.engram_prompt_attention(cache, q, P.dev(np.arange(6)), P.dev(table), P.dev(lens), lse=True, **how)
            assert float((a.float() - b.float()).abs().max()) < 2.0 ** -5
            assert torch.equal(torch.isneginf(la), torch.isneginf(lb))
            assert float((la - lb).nan_to_num(0.0).abs().max()) < 1e-4


def test_one_workspace_for_every_attention_call_in_order():
    """Calls of different shapes share a workspace, and leave its start zero; each repeats itself bit for bit."""
    E = H.pkg()
    lens = [2000, 31, 700]
    cache, table = H.filled(lens, 16, 2, 128, "bf16", 23)
    wide, wtable = H.filled([900], 32, 1, 256, "fp8", 24)
    size = max(E.prompt_workspace_bytes(cache, 8, 600, 3), E.prompt_workspace_bytes(wide, 4, 300, 1),
               E.attention_workspace_bytes(cache, 8, 3), E.shared_workspace_bytes(cache, 8, 3, 1))
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    ws[:ZERO] = 0
    q, qw, q1 = randn(25, (600, 8, 128)), randn(26, (300, 4, 256)), randn(27, (3, 8, 128))
    calls = [lambda **k: E.engram_prompt_attention(cache, q, P.dev([0, 500, 520, 600]), P.dev(table), P.dev(lens), lse=True, **k),
             lambda **k: E.engram_prompt_attention(wide, qw, P.dev([0, 300]), P.dev(wtable), P.dev([900]), lse=True, **k),
             lambda **k: E.engram_paged_attention(cache, q1, P.dev(table), P.dev(lens), lse=True, **k),
             lambda **k: E.engram_shared_attention(cache, q1, P.dev(table[:1]), P.dev([2000]), P.dev([0, 3]), P.dev(table[1:2]).expand(3, -1).contiguous(),
                                                   P.dev([31, 7, 0]), lse=True, **k)]
    first = [c(workspace=ws) for c in calls]
    assert not ws[:ZERO].any()
    for i in (3, 0, 2, 1, 0, 3):
        got = calls[i](workspace=ws)
        assert torch.equal(got[0], first[i][0]) and torch.equal(got[1], first[i][1])
    alone = [c() for c in calls]
    for a, b in zip(first, alone):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_replayed_and_on_other_streams():
    E = H.pkg()
    lens, new = [1500, 20, 333], [400, 20, 1]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 28)
    q = randn(29, (421, 8, 64))
    cu, bt, sl = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    plan = E.PromptAttentionPlan(cache, q, cu, bt, sl, lse=True)
    plan.run()
    want = plan.out.clone(), plan.lse.clone()
    P.check_prompt(cache, table, new, lens, q, *want, 64 ** -0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
        plan.run()
    for new2, lens2 in ((new, lens), ([1, 20, 400], [900, 20, 333]), ([0, 0, 0], lens)):   # other lengths, the same graph
        cu.copy_(P.dev(cu_of(new2)))
        sl.copy_(P.dev(lens2))
        plan.out.fill_(9.0)
        plan.lse.fill_(9.0)
        graph.replay()
        T2 = sum(new2)
        P.check_prompt(cache, table, new2, lens2, q[:T2], plan.out[:T2], plan.lse[:T2], 64 ** -0.5)
        assert bool((plan.out[T2:] == 9).all())
    cu.copy_(P.dev(cu_of(new)))
    sl.copy_(P.dev(lens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.out.fill_(9.0)
    side.wait_stream(torch.cuda.current_stream())
    plan.run(side)
    side.synchronize()
    assert torch.equal(plan.out, want[0]) and torch.equal(plan.lse, want[1])


def test_two_calls_at_once_with_workspaces_of_their_own():
    E = H.pkg()
    lens, new = [3000, 400], [300, 400]
    cache, table = H.filled(lens, 16, 2, 128, "bf16", 30)
    q = randn(31, (700, 8, 128))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    want = E.engram_prompt_attention(cache, q, *args)
    streams = [torch.cuda.Stream() for _ in range(3)]
    plans = [E.PromptAttentionPlan(cache, q, *args) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, p in zip(streams, plans):
            p.run(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p.out, want) for p in plans)


def test_offsets_past_32_bits():
    """Pages further apart than 2^32 bytes altogether, and a head far from its page's start."""
    E, page, Hk, D = H.pkg(), 16, 2, 64
    pages, stride = 40, 2 ** 27                              # 40 pages of 256 MB apart: 10 GB
    buf = torch.empty(pages * stride, dtype=torch.bfloat16, device=DEV)
    # key rows first, value rows 4 KB behind; heads 2^26 values apart
    k = torch.as_strided(buf, (pages, Hk, page, D), (stride, 2 ** 26, D, 1))
    v = torch.as_strided(buf, (pages, Hk, page, D), (stride, 2 ** 26, D, 1), 2048)
    cache = E.KVCache(k, v)
    lens, new = [600], [130]
    table = np.random.default_rng(1).permutation(pages)[None, :38].astype(np.int32)
    slots = H.slots_of(table, 0, 0, 600, page)
    E.engram_kv_write(cache, randn(1, (600, Hk, D)), randn(2, (600, Hk, D)), torch.from_numpy(slots).to(DEV))
    q = randn(3, (130, 8, D))
    out, lse = E.engram_prompt_attention(cache, q, P.dev([0, 130]), P.dev(table), P.dev(lens), lse=True)
    P.check_prompt(cache, table, new, lens, q, out, lse, D ** -0.5)


def test_many_sequences_and_long_ones():
    """More sequences than a block has threads, most of them idle; one of 20000 tokens among them."""
    E = H.pkg()
    B = 1500
    rng = np.random.default_rng(5)
    new = np.where(rng.random(B) < 0.1, rng.integers(1, 9, B), 0)
    old = rng.integers(0, 40, B)
    new[700], old[700] = 200, 19800
    new, lens = new.tolist(), (new + old).tolist()
    cache, table = H.filled(lens, 16, 1, 64, "bf16", 32)
    T = sum(new)
    q = randn(33, (T, 4, 64))
    out, lse = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), lse=True)
    P.check_prompt(cache, table, new, lens, q, out, lse, 64 ** -0.5)




@pytest.mark.parametrize("slopes", [False, True])
def test_pairs_of_tiles_and_single_ones_in_turn(slopes):
    """Sequences of many lengths in one batch: a block goes from two tiles of rows to one and back, with key tiles of any
    number in between, and several times over."""
    E = H.pkg()
    new = [113, 2011, 60, 700, 1, 333, 1290, 129, 97, 512, 40, 257] * 2
    cache, table = H.filled(new, 24, 4, 64, "bf16", 40)
    T = sum(new)
    q = randn(41, (T, 4, 64))
    sl = P.alibi(4) if slopes else None
    err = word()
    for _ in range(3):
        out, lse = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(new), lse=True, err=err,
                                             slopes=None if sl is None else P.dev(sl, torch.float32))
    assert int(err) == 0
    P.check_prompt(cache, table, new, new, q, out, lse, 64 ** -0.5, slopes=sl)


def test_few_new_tokens_over_long_caches_many_times():
    """Drafted tokens: one tile of rows, key tiles that are cut between blocks, and nothing behind a sequence's last key that
    may be used. Every call gives the same bits."""
    E = H.pkg()
    new, lens = [5] * 32, [1024 + 97 * b for b in range(32)]
    cache, table = H.filled(lens, 64, 8, 128, "bf16", 42)
    q = randn(43, (160, 32, 128))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    ws, err = E.prompt_workspace(cache, 32, 160, 32), word()
    out, lse = E.engram_prompt_attention(cache, q, *args, lse=True, workspace=ws, err=err)
    P.check_prompt(cache, table, new, lens, q, out, lse, 128 ** -0.5)
    for _ in range(30):
        again = E.engram_prompt_attention(cache, q, *args, lse=True, workspace=ws, err=err)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert int(err) == 0


@pytest.mark.parametrize("D,cap,slopes,fmt", [(128, 0.0, False, "bf16"), (64, 0.0, True, "bf16"), (128, 30.0, False, "bf16"), (192, 0.0, False, "fp8"),
                                              (128, 50.0, True, "fp8"), (256, 300.0, False, "bf16")])
def test_a_token_that_sees_one_key_gives_its_value(D, cap, slopes, fmt):
    """The only weight is 1 up to 2^-18 (of scores up to 2^6), so that a value that bf16 holds comes out as it is."""
    E = H.pkg()
    new = [300, 1, 77]
    cache, table = H.filled(new, 16, 2, D, fmt, 44)
    q = randn(45, (378, 8, D))
    at = np.concatenate([np.arange(n) for n in new])
    args = dict(cap=cap, slopes=P.dev(P.alibi(8), torch.float32) if slopes else None)
    out = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(new), doc_starts=P.dev(at), **args)
    values = np.concatenate([P.rows_of(cache, table, b, n)[1] for b, n in enumerate(new)])
    assert np.array_equal(out.double().cpu().numpy(), np.repeat(values, 4, axis=1))


@pytest.mark.parametrize("new,old,page,Hq,Hk,D,mask", [
    ([300], [40], 5, 8, 2, 128, "docs"), ([130, 7, 260], [0, 500, 3], 12, 3, 3, 192, "causal"), ([515], [100], 1, 4, 1, 64, "window"),
    ([200, 90], [0, 700], 20, 16, 2, 256, "prefix")])
def test_fp8_pages_that_do_not_divide_into_boxes(new, old, page, Hq, Hk, D, mask):
    test_prompts_match_the_formula(new, old, page, Hq, Hk, D, "fp8", "hnd", mask, 0.0, False)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D,page", [(128, 64), (256, 16), (256, 5), (160, 32), (128, 6)])
def test_values_that_are_not_finite_stay_with_those_that_see_them(fmt, D, page):
    """Heads of one and of two tiles, boxes and rows, work that is cut between CTAs: NaN in one position of some values."""
    E, new, lens = H.pkg(), [700, 333], [700, 1000]
    cache, table = H.filled(lens, page, 2, D, fmt, 46)
    q = randn(47, (1033, 8, D))
    args = P.dev(cu_of(new)), P.dev(table), P.dev(lens)
    doc = documents(new, lens, 60, 5)
    how = dict(doc_starts=P.dev(doc), lse=True)
    want, want_lse = E.engram_prompt_attention(cache, q, *args, **how)
    P.check_prompt(cache, table, new, lens, q, want, want_lse, D ** -0.5, doc_starts=doc)
    bad = {0: [0, 90, 311, 640], 1: [667, 800, 999]}
    at = D - 3
    for b, keys in bad.items():
        for j in keys:
            s = H.slots_of(table, b, j, j + 1, page)[0]
            cache.v[s // page, :, s % page, at] = float("nan") if fmt == "bf16" else 0x7F
    out, lse = E.engram_prompt_attention(cache, q, *args, **how)
    hit, t0 = np.zeros(1033, bool), 0
    for b, (n, m) in enumerate(zip(new, lens)):
        for i in range(n):
            hit[t0 + i] = any(doc[t0 + i] <= j <= m - n + i for j in bad[b])
        t0 += n
    assert 50 < hit.sum() < 1000
    hit = torch.from_numpy(hit).to(DEV)
    assert torch.equal(lse, want_lse)
    assert torch.isnan(out[hit][..., at]).all()
    assert torch.equal(out[~hit], want[~hit])
    rest = [d for d in range(D) if d != at]
    # the other positions of rows that see one: its products are added one by one, in another order of fp32 sums
    assert torch.isfinite(out[hit][..., rest]).all()
    assert float((out[hit][..., rest].double() - want[hit][..., rest].double()).abs().max()) <= 2.0 ** -7 * float(want.double().abs().max())


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_that_are_not_positive(scale):
    E, new, lens = H.pkg(), [300], [420]
    cache, table = H.filled(lens, 16, 2, 128, "bf16", 48)
    q = randn(49, (300, 8, 128))
    out, lse = E.engram_prompt_attention(cache, q, P.dev(cu_of(new)), P.dev(table), P.dev(lens), scale=scale, lse=True)
    P.check_prompt(cache, table, new, lens, q, out, lse, scale)
