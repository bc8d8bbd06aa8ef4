"""Forms of scores for single tokens, and batches whose sequences share a prefix, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests import _attention as H
from tests import _prompts as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
ZERO = 16384


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def randn(seed, shape, std=1.0, dtype=torch.bfloat16):
    return (std * torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)).to(dtype)


# ------------------------------------------------------------------------------------------ single tokens

def check_tokens(cache, table, lens, q, out, lse, scale, window, cap, slopes):
    for b, n in enumerate(lens):
        k, v = P.rows_of(cache, table, b, n)
        p, lo, hi = A.visible(1, n, True, window)
        seen = (np.arange(n) >= lo[:, None]) & (np.arange(n) < hi[:, None])
        ref = A.attention_rows(q[b:b + 1].double().cpu().numpy(), k, v, seen, p, scale, cap, slopes, H.Q_REL[cache.fmt, q.dtype],
                               H.P_REL[cache.fmt])
        P.check_rows(out[b:b + 1].double().cpu().numpy(), lse[b:b + 1].double().cpu().numpy(), ref, f"sequence {b} of {n}")


@pytest.mark.parametrize("cap,slopes,window", [(30.0, False, 0), (0.0, True, 0), (8.0, True, 200)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hk,D,page,dtype", [(8, 2, 128, 16, "bf16"), (8, 2, 128, 64, "f32"), (3, 3, 64, 24, "bf16"), (32, 2, 64, 16, "f32"),
                                                (12, 1, 256, 32, "bf16"), (5, 1, 256, 16, "f32"), (40, 2, 96, 7, "bf16"), (4, 4, 192, 16, "bf16")])
def test_single_tokens_with_a_form_match_the_formula(Hq, Hk, D, page, dtype, fmt, cap, slopes, window):
    E, lens = H.pkg(), [1, 0, 900, 17, 3001, 250]
    cache, table = H.filled(lens, page, Hk, D, fmt, D + Hq)
    q = randn(Hq, (len(lens), Hq, D), cap / 4 if cap else 1.5, torch.bfloat16 if dtype == "bf16" else torch.float32)
    sl = P.alibi(Hq) if slopes else None
    ws, err = E.attention_workspace(cache, Hq, 0), word()
    out, lse = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), window=window, lse=True, cap=cap, workspace=ws, err=err,
                                        slopes=None if sl is None else P.dev(sl, torch.float32))
    assert int(err) == 0 and not ws[:ZERO].any()
    check_tokens(cache, table, lens, q, out, lse, D ** -0.5, window, cap, sl)


def test_more_than_32_sequences_and_a_long_one_with_a_form():
    E = H.pkg()
    lens = [37 * i % 800 for i in range(70)] + [30000]
    cache, table = H.filled(lens, 16, 2, 64, "bf16", 1)
    q = randn(2, (71, 8, 64), 3.0)
    out, lse = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), lse=True, cap=10.0, slopes=P.dev(P.alibi(8), torch.float32))
    check_tokens(cache, table, lens, q, out, lse, 64 ** -0.5, 0, 10.0, P.alibi(8))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_forms_without_effect_change_nothing(fmt):
    """Slopes of zero and a cap of 2^60 leave scores as they are, but for a rounding of their own (over FP8 a score and its
    row's scale are otherwise joined in one fused multiply-add)."""
    E, lens = H.pkg(), [5, 700, 64]
    cache, table = H.filled(lens, 16, 2, 128, fmt, 3)
    q = randn(4, (3, 8, 128))
    b = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), lse=True, slopes=torch.zeros(8, device=DEV))
    check_tokens(cache, table, lens, q, *b, 128 ** -0.5, 0, 0.0, None)
    c = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), lse=True, cap=2.0 ** 60)
    check_tokens(cache, table, lens, q, *c, 128 ** -0.5, 0, 2.0 ** 60, None)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("cap,slopes", [(20.0, False), (0.0, True), (15.0, True)])
def test_a_step_with_a_form_equals_its_parts(fmt, cap, slopes):
    E, lens, Hq, Hk, D = H.pkg(), [1, 40, 700, 333], 8, 2, 128
    caches = [H.filled(lens, 16, Hk, D, fmt, 5) for _ in range(2)]
    table = caches[0][1]
    g = torch.Generator(device=DEV).manual_seed(6)
    w = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2)]
    nr = E.NormRope(*w, 1e-6, E.rope_table(1024, D))
    q, k, v = (randn(7 + i, (4, h, D), 2.0) for i, h in enumerate((Hq, Hk, Hk)))
    pos = P.dev([n - 1 for n in lens])
    slots = torch.tensor([H.slots_of(table, b, n - 1, n, 16)[0] for b, n in enumerate(lens)], device=DEV)
    form = dict(cap=cap, slopes=P.dev(P.alibi(Hq), torch.float32) if slopes else None)
    a = E.engram_attention_step(nr, caches[0][0], q, k, v, pos, slots, P.dev(table), P.dev(lens), lse=True, **form)
    turned = [torch.empty(x.shape, dtype=torch.float32, device=DEV) for x in (q, k)]
    E.engram_qk_norm_rope(nr, q, k, pos, *turned)
    E.engram_kv_write(caches[1][0], turned[1], v.float(), slots)
    b = E.engram_paged_attention(caches[1][0], turned[0], P.dev(table), P.dev(lens), lse=True, **form)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(caches[0][0].k, caches[1][0].k) or fmt == "bf16"     # NaN outside of the tokens in bf16


# ---------------------------------------------------------------------------------------- shared prefixes

def setup(groups, prefix, lens, page, Hk, D, fmt, seed, layout="hnd"):
    """A cache that holds the prefixes and then the sequences' own tokens; both page tables."""
    cache, table = H.filled([*prefix, *lens], page, Hk, D, fmt, seed, layout)
    n = len(prefix)
    return cache, table[:n], table[n:]


def check_shared(cache, ptable, table, groups, prefix, lens, q, out, lse, scale, cap=0.0, slopes=None):
    starts = np.concatenate([[0], np.cumsum(groups)])
    for b, n in enumerate(lens):
        g = int(np.searchsorted(starts, b, side="right")) - 1
        m = prefix[g] if g < len(prefix) else 0
        k, v = P.rows_of(cache, table, b, n)
        if m:
            k, v = (np.concatenate(x) for x in zip(P.rows_of(cache, ptable, g, m), (k, v)))
        seen = np.ones((1, m + n), bool)
        # the prefix's weights are rounded to bf16, and both parts' fp32 sums are joined by weights off by 2^-20
        ref = A.attention_rows(q[b:b + 1].double().cpu().numpy(), k, v, seen, [m + n - 1], scale, cap, slopes,
                               p_rel=max(P.P_PROMPT, H.P_REL[cache.fmt]) + 2.0 ** -20)
        P.check_rows(out[b:b + 1].double().cpu().numpy(), lse[b:b + 1].double().cpu().numpy(), ref, f"sequence {b}: {m} and {n}")


SHARED = [
    # groups, prefixes, own tokens, page, Hq, Hk, D, cache, layout, cap, slopes
    ([1], [1], [1], 16, 4, 1, 64, "bf16", "hnd", 0.0, False),
    ([4], [500], [1, 64, 7, 0], 16, 32, 8, 128, "bf16", "hnd", 0.0, False),
    ([33], [1500], [(i * 37) % 200 for i in range(33)], 64, 16, 2, 128, "bf16", "nhd", 0.0, True),
    ([70], [260], [1] * 70, 24, 8, 2, 96, "bf16", "hnd", 12.0, False),
    ([3, 0, 9, 1, 5], [300, 77, 0, 1025, 64], [(i * 53) % 90 for i in range(18)], 16, 8, 4, 64, "bf16", "hnd", 0.0, False),
    ([3, 0, 9, 1, 5], [300, 77, 0, 1025, 64], [(i * 53) % 90 for i in range(18)], 16, 8, 1, 128, "fp8", "padded", 20.0, True),
    ([6, 20], [2000, 130], [(i * 31) % 400 for i in range(26)], 32, 12, 1, 256, "bf16", "hnd", 0.0, False),
    ([6, 20], [2000, 130], [(i * 31) % 400 for i in range(26)], 32, 5, 5, 192, "fp8", "hnd", 0.0, False),
]


@pytest.mark.parametrize("groups,prefix,lens,page,Hq,Hk,D,fmt,layout,cap,slopes", SHARED)
def test_shared_prefixes_match_the_formula(groups, prefix, lens, page, Hq, Hk, D, fmt, layout, cap, slopes):
    E, B = H.pkg(), len(lens)
    cache, ptable, table = setup(groups, prefix, lens, page, Hk, D, fmt, B + D, layout)
    q = randn(B, (B, Hq, D), cap / 4 if cap else 1.5)
    sl = P.alibi(Hq) if slopes else None
    ws, err = E.shared_workspace(cache, Hq, B, len(groups)), word()
    ws[ZERO:] = 0xFF                                          # NaN: nothing is read that the call has not written
    out, lse = E.engram_shared_attention(cache, q, P.dev(ptable), P.dev(prefix), P.dev(np.concatenate([[0], np.cumsum(groups)])),
                                         P.dev(table), P.dev(lens), cap=cap, slopes=None if sl is None else P.dev(sl, torch.float32),
                                         lse=True, workspace=ws, err=err)
    assert int(err) == 0 and not ws[:ZERO].any()
    check_shared(cache, ptable, table, groups, prefix, lens, q, out, lse, D ** -0.5, cap, sl)


def test_sequences_in_no_group_have_no_prefix():
    E, lens, prefix = H.pkg(), [10, 200, 0, 33, 64, 5], [400]
    cache, ptable, table = setup([3], prefix, lens, 16, 2, 64, "bf16", 8)
    q = randn(9, (6, 8, 64))
    out, lse = E.engram_shared_attention(cache, q, P.dev(ptable), P.dev(prefix), P.dev([1, 4]), P.dev(table), P.dev(lens), lse=True)
    alone = E.engram_paged_attention(cache, q, P.dev(table), P.dev(lens), lse=True)
    for b in (0, 4, 5):
        assert float((out[b].float() - alone[0][b].float()).abs().max()) <= 2.0 ** -7
        assert float((lse[b] - alone[1][b]).abs().max()) <= 1e-5
    check_shared(cache, ptable, table[1:4], [3], prefix, lens[1:4], q[1:4], out[1:4], lse[1:4], 64 ** -0.5)
    none = E.engram_shared_attention(cache, q, P.dev(ptable[:0]), P.dev(np.zeros(0)), P.dev([0]), P.dev(table), P.dev(lens), lse=True)
    for b in (0, 1, 3, 4, 5):
        assert float((none[0][b].float() - alone[0][b].float()).abs().max()) <= 2.0 ** -7
    assert not none[0][2].any() and bool(torch.isneginf(none[1][2]).all())


def test_a_view_of_whole_page_tables():
    """The prefix's pages stand first in every sequence's table: the own part is a view behind them."""
    E, page, m, lens = H.pkg(), 16, 320, [1, 100, 17, 240]
    cache, ptable, table = setup([4], [m], lens, page, 2, 128, "fp8", 10)
    whole = np.concatenate([np.repeat(ptable[:, :m // page], 4, 0), table[:, :-(-max(lens) // page)]], 1)
    wt, q = P.dev(whole), randn(11, (4, 8, 128))
    out, lse = E.engram_shared_attention(cache, q, wt[:1], P.dev([m]), P.dev([0, 4]), wt[:, m // page:], P.dev(lens), lse=True)
    check_shared(cache, ptable, table, [4], [m], lens, q, out, lse, 128 ** -0.5)
    plain, plain_lse = E.engram_paged_attention(cache, q, wt, P.dev([m + n for n in lens]), lse=True)
    assert float((out.float() - plain.float()).abs().max()) < 2.0 ** -5 and float((lse - plain_lse).abs().max()) < 1e-4


def test_starts_lengths_and_pages_that_do_not_fit():
    E, lens, prefix = H.pkg(), [10, 20, 30], [200]
    cache, ptable, table = setup([3], prefix, lens, 16, 2, 64, "bf16", 12)
    q = randn(13, (3, 4, 64))
    want = E.engram_shared_attention(cache, q, P.dev(ptable), P.dev(prefix), P.dev([0, 3]), P.dev(table), P.dev(lens), lse=True)
    for starts, m in (([-4, 3], 200), ([0, 99], 200)):
        err = word()
        got = E.engram_shared_attention(cache, q, P.dev(ptable), P.dev([m]), P.dev(starts), P.dev(table), P.dev(lens), lse=True, err=err)
        assert int(err) == E.ERR_SEQ_LEN and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    err = word()
    lost = ptable.copy()
    lost[0, 2] = -9
    out, lse = E.engram_shared_attention(cache, q, P.dev(lost), P.dev(prefix), P.dev([0, 3]), P.dev(table), P.dev(lens), lse=True, err=err)
    assert int(err) == E.ERR_PAGE
    for b, n in enumerate(lens):
        k, v = (np.concatenate(x) for x in zip(P.rows_of(cache, ptable, 0, 200), P.rows_of(cache, table, b, n)))
        seen = np.ones((1, 200 + n), bool)
        seen[:, 32:48] = False
        ref = A.attention_rows(q[b:b + 1].double().cpu().numpy(), k, v, seen, [199 + n], 64 ** -0.5, p_rel=P.P_PROMPT + 2.0 ** -20)
        P.check_rows(out[b:b + 1].double().cpu().numpy(), lse[b:b + 1].double().cpu().numpy(), ref, f"sequence {b}")


def test_strides_capture_and_other_streams():
    E, lens, prefix = H.pkg(), [10, 200, 0, 33, 64], [400, 90]
    cache, ptable, table = setup([3, 2], prefix, lens, 16, 2, 64, "bf16", 14)
    rows = randn(15, (5, 12, 64))
    q = rows[:, 2:10]
    out = torch.full((8, 5, 64), float("nan"), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    pl, gs, sl = P.dev(prefix), P.dev([0, 3, 5]), P.dev(lens)
    plan = E.SharedAttentionPlan(cache, q, P.dev(ptable), pl, gs, P.dev(table), sl, out=out, lse=True)
    plan.run()
    check_shared(cache, ptable, table, [3, 2], prefix, lens, q, out, plan.lse, 64 ** -0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    lens2, prefix2 = [9, 0, 0, 30, 1], [17, 0]
    sl.copy_(P.dev(lens2))
    pl.copy_(P.dev(prefix2))
    gs.copy_(P.dev([0, 4, 5]))
    out.fill_(float("nan"))
    graph.replay()
    check_shared(cache, ptable, table, [4, 1], prefix2, lens2, q, out, plan.lse, 64 ** -0.5)
    want = out.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    plan.run(side)
    side.synchronize()
    assert torch.equal(out, want)


def test_prompts_then_tokens_then_shared_answers_of_one_layer():
    """A run of them as a program has it: a prompt goes through, its last tokens are drafted again, answers branch off it."""
    E, Hq, Hk, D, page = H.pkg(), 8, 2, 128, 16
    for fmt in ("bf16", "fp8"):
        n, B = 320, 5
        cache = H.empty_cache(60, page, Hk, D, fmt)
        rng = np.random.default_rng(16)
        places = rng.permutation(60)
        prompt = places[None, :n // page].astype(np.int32)
        own = places[n // page:n // page + B * 2].reshape(B, 2).astype(np.int32)
        rows = [randn(17 + i, (n, h, D)) for i, h in enumerate((Hq, Hk, Hk))]
        slots = H.slots_of(prompt, 0, 0, n, page)
        E.engram_kv_write(cache, rows[1], rows[2], torch.from_numpy(slots).to(DEV))
        out, lse = E.engram_prompt_attention(cache, rows[0], P.dev([0, n]), P.dev(prompt), P.dev([n]), lse=True, cap=25.0)
        P.check_prompt(cache, prompt, [n], [n], rows[0], out, lse, D ** -0.5, cap=25.0)
        # the same in two chunks gives the same rows to the weights' rounding
        tail = E.engram_prompt_attention(cache, rows[0][200:], P.dev([0, n - 200]), P.dev(prompt), P.dev([n]), cap=25.0)
        assert float((tail.float() - out[200:].float()).abs().max()) < 2.0 ** -5
        # answers of their own lengths behind the prompt
        lens = [1, 7, 24, 16, 17]
        whole = np.concatenate([np.repeat(prompt, B, 0), own], 1)
        for b, m in enumerate(lens):
            s = torch.from_numpy(H.slots_of(own, b, 0, m, page)).to(DEV)
            E.engram_kv_write(cache, randn(30 + b, (m, Hk, D)), randn(40 + b, (m, Hk, D)), s)
        q = randn(50, (B, Hq, D))
        a, la = E.engram_shared_attention(cache, q, P.dev(prompt), P.dev([n]), P.dev([0, B]), P.dev(own), P.dev(lens), lse=True, cap=25.0)
        check_shared(cache, prompt, own, [B], [n], lens, q, a, la, D ** -0.5, 25.0)
        c, lc = E.engram_paged_attention(cache, q, P.dev(whole), P.dev([n + m for m in lens]), lse=True, cap=25.0)
        assert float((a.float() - c.float()).abs().max()) < 2.0 ** -5 and float((la - lc).abs().max()) < 1e-4
