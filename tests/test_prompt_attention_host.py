"""Prompts, forms of scores and shared prefixes without a GPU: their refusals (shapes and types in the binding, pointers,
strides and sizes in the C ABI, each before any CUDA call) and the pins of their 64-bit oracle."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests.test_attention_host import Abi, E  # noqa: F401

T_, B_, G_, HQ, HK, D, PAGE, PAGES = 7, 3, 2, 4, 2, 64, 16, 10
I32 = torch.int32


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _good(E, fn, fmt="bf16"):
    cache = E.KVCache.allocate(PAGES, PAGE, HK, D, fmt, device="cpu")
    a = dict(cache=cache, q=_z(B_, HQ, D), block_table=_z(B_, 4, dtype=I32), seq_lens=_z(B_, dtype=I32))
    if fn == "engram_prompt_attention":
        a |= dict(q=_z(T_, HQ, D), cu_seqlens=_z(B_ + 1, dtype=I32))
    if fn == "engram_shared_attention":
        a |= dict(prefix_table=_z(G_, 6, dtype=I32), prefix_lens=_z(G_, dtype=I32), groups=_z(G_ + 1, dtype=I32))
    return a


def _call(E, fn, a, **more):
    return getattr(E, fn)(**a, **more)


FNS = ("engram_prompt_attention", "engram_shared_attention", "engram_paged_attention")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("fn", FNS)
def test_well_formed_cpu_tensors_are_refused_for_their_device_only(E, fn, fmt):
    with pytest.raises(ValueError, match="CUDA"):
        _call(E, fn, _good(E, fn, fmt), cap=30.0, slopes=_z(HQ, dtype=torch.float32))


P, S = "engram_prompt_attention", "engram_shared_attention"


@pytest.mark.parametrize("fn,name,make,words", [
    (P, "q", lambda: _z(T_, HQ, D, dtype=torch.float32), "q must be"),
    (P, "q", lambda: _z(T_, HQ * D), "dimensions"),
    (P, "q", lambda: _z(T_, HQ, 2 * D), "heads of"),
    (P, "q", lambda: _z(T_, HK + 1, D), "multiple"),
    (P, "cu_seqlens", lambda: _z(B_, dtype=I32), "block_table"),
    (P, "cu_seqlens", lambda: _z(B_ + 1, dtype=torch.int64), "cu_seqlens"),
    (P, "cu_seqlens", lambda: _z(2 * B_ + 2, dtype=I32)[::2], "contiguous"),
    (P, "cu_seqlens", lambda: _z(0, dtype=I32), "cu_seqlens"),
    (P, "cu_seqlens", lambda: None, "cu_seqlens"),
    (P, "block_table", lambda: _z(B_, 4, dtype=torch.int64), "block_table"),
    (P, "block_table", lambda: _z(4, B_, dtype=I32).T, "contiguous"),
    (P, "block_table", lambda: _z(4 + B_, dtype=I32).as_strided((B_, 4), (1, 1)), "overlap"),
    (P, "seq_lens", lambda: _z(B_ + 1, dtype=I32), "seq_lens"),
    (P, "seq_lens", lambda: None, "seq_lens"),
    (S, "q", lambda: _z(B_, HQ, D, dtype=torch.float32), "q must be"),
    (S, "q", lambda: _z(B_ + 1, HQ, D), "block_table"),
    (S, "groups", lambda: _z(G_ + 2, dtype=I32), "prefix_table"),
    (S, "groups", lambda: _z(G_ + 1, dtype=torch.int64), "groups"),
    (S, "groups", lambda: _z(0, dtype=I32), "groups"),
    (S, "prefix_table", lambda: _z(G_, 6, dtype=torch.int64), "prefix_table"),
    (S, "prefix_lens", lambda: _z(G_ + 1, dtype=I32), "prefix_lens"),
    (S, "prefix_lens", lambda: None, "prefix_lens"),
    (S, "seq_lens", lambda: _z(B_, dtype=torch.int64), "seq_lens"),
])
def test_the_binding_refuses(E, fn, name, make, words):
    a = _good(E, fn)
    a[name] = make()
    with pytest.raises((ValueError, TypeError), match=words):
        _call(E, fn, a)


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("more,words", [
    (dict(cap=-1.0), "cap"), (dict(cap=math.nan), "cap"), (dict(cap=math.inf), "cap"), (dict(cap=2.0 ** -61), "cap"),
    (dict(slopes=_z(HQ)), "slopes"), (dict(slopes=_z(HQ + 1, dtype=torch.float32)), "slopes"),
    (dict(slopes=_z(2 * HQ, dtype=torch.float32)[::2]), "contiguous"), (dict(slopes=1.0), "slopes"),
    (dict(lse=3), "lse"), (dict(lse=_z(2, HQ, dtype=torch.float32)), "lse"), (dict(out=_z(2, HQ, D)), "out"),
    (dict(out=_z(B_, HQ, D, dtype=torch.float32)), "out"), (dict(workspace=_z(64)), "workspace"), (dict(err=_z(1)), "err"),
])
def test_the_binding_refuses_forms_and_outputs(E, fn, more, words):
    with pytest.raises((ValueError, TypeError), match=words):
        _call(E, fn, _good(E, fn), **more)


@pytest.mark.parametrize("more,words", [
    (dict(window=-1), "window"), (dict(doc_starts=_z(T_ + 1, dtype=I32)), "doc_starts"),
    (dict(doc_starts=_z(T_, dtype=torch.int64)), "doc_starts"), (dict(prefix_ends=_z(B_, dtype=I32)), "prefix_ends"),
    (dict(prefix_ends=_z(T_, dtype=I32), causal=False), "causal"),
])
def test_the_binding_refuses_masks_of_prompts(E, more, words):
    with pytest.raises((ValueError, TypeError), match=words):
        _call(E, P, _good(E, P), **more)


# --------------------------------------------------------------------------------------- the C ABI

class Abi2(Abi):
    def form(self, cap=30.0, slopes=True):
        return C.byref(self.M._Scores(cap, self.p if slopes is True else slopes))

    def attend2(self, scores=None):
        h = self.heads()
        return self.L.engram_paged_attention2(C.byref(self.cache()), C.byref(self.seqs()), C.byref(h), 0.1, 0, scores, C.byref(h), None,
                                              self.p, 1 << 40, None, None)

    def step2(self, scores=None):
        h = [C.byref(self.heads()) for _ in range(3)]
        return self.L.engram_attention_step2(C.byref(self.nr()), C.byref(self.cache()), C.byref(self.seqs()), *h, self.p, self.p, 0.1, 0,
                                             scores, C.byref(self.heads()), None, self.p, 1 << 40, None, None)

    def prompt(self, cache=None, seqs=None, T=2, cu=True, q=None, scale=0.1, visible=True, scores=None, out=None, lse=None, ws=True,
               n=1 << 40):
        v = self.M._Visible(1, 0, None, None) if visible is True else visible
        return self.L.engram_prompt_attention(C.byref(cache or self.cache()), C.byref(seqs or self.seqs()), T, self.p if cu is True else cu,
                                              C.byref(q or self.heads()), scale, None if v is None else C.byref(v), scores,
                                              C.byref(out or self.heads()), lse, self.p if ws is True else ws, n, None, None)

    def shared(self, cache=None, prefix=None, groups=True, seqs=None, q=None, scale=0.1, scores=None, out=None, lse=None, ws=True,
               n=1 << 40):
        return self.L.engram_shared_attention(C.byref(cache or self.cache()), C.byref(prefix or self.seqs()),
                                              self.p if groups is True else groups, C.byref(seqs or self.seqs()), C.byref(q or self.heads()),
                                              scale, scores, C.byref(out or self.heads()), lse, self.p if ws is True else ws, n, None, None)


def _visible(a, **kw):
    v = a.M._Visible(1, 0, None, None)
    for n, x in kw.items():
        setattr(v, n, x)
    return v


ABI_REFUSALS = [
    (lambda a: a.attend2(a.form(-1.0)), "cap"), (lambda a: a.attend2(a.form(math.nan)), "cap"), (lambda a: a.attend2(a.form(2.0 ** 61)), "cap"),
    (lambda a: a.attend2(a.form(0.0, a.p + 2)), "slopes"), (lambda a: a.step2(a.form(math.inf)), "cap"),
    (lambda a: a.step2(a.form(1.0, a.p + 1)), "slopes"),
    (lambda a: a.prompt(cache=a.cache(page_size=0)), "page_size"), (lambda a: a.prompt(T=-1), "T must"),
    (lambda a: a.prompt(T=1 << 31), "T must"), (lambda a: a.prompt(T=1 << 30, q=a.heads(heads=4, ts=256), out=a.heads(heads=4, ts=256)), "2^31"),
    (lambda a: a.prompt(cu=None), "cu_seqlens"), (lambda a: a.prompt(cu=a.p + 2), "cu_seqlens"),
    (lambda a: a.prompt(seqs=a.seqs(batch=-1)), "batch"), (lambda a: a.prompt(seqs=a.seqs(table_stride=3)), "stride"),
    (lambda a: a.prompt(seqs=a.seqs(block_table=None)), "block_table"), (lambda a: a.prompt(seqs=a.seqs(seq_lens=a.p + 2)), "seq_lens"),
    (lambda a: a.prompt(q=a.heads(type=1)), "bf16"), (lambda a: a.prompt(q=a.heads(heads=3)), "multiple"),
    (lambda a: a.prompt(q=a.heads(data=a.p + 8)), "16 bytes"), (lambda a: a.prompt(q=a.heads(ts=132)), "16 bytes"),
    (lambda a: a.prompt(scale=math.nan), "scale"), (lambda a: a.prompt(scale=-math.inf), "scale"),
    (lambda a: a.prompt(visible=None), "visible"), (lambda a: a.prompt(visible=_visible(a, window=-1)), "window"),
    (lambda a: a.prompt(visible=_visible(a, doc_starts=a.p + 1)), "doc_starts"),
    (lambda a: a.prompt(visible=_visible(a, causal=0, prefix_ends=a.p)), "causal"),
    (lambda a: a.prompt(scores=a.form(-2.0)), "cap"), (lambda a: a.prompt(out=a.heads(type=1)), "out"),
    (lambda a: a.prompt(out=a.heads(heads=4, ts=256)), "out"), (lambda a: a.prompt(out=a.heads(ts=64)), "overlap"),
    (lambda a: a.prompt(lse=a.p + 2), "lse"), (lambda a: a.prompt(ws=None), "workspace"), (lambda a: a.prompt(ws=a.p + 128), "workspace"),
    (lambda a: a.prompt(n=16384), "workspace"),
    (lambda a: a.shared(prefix=a.seqs(batch=-1)), "batch"), (lambda a: a.shared(prefix=a.seqs(block_table=None)), "block_table"),
    (lambda a: a.shared(groups=None), "group_starts"), (lambda a: a.shared(groups=a.p + 1), "group_starts"),
    (lambda a: a.shared(q=a.heads(type=1)), "bf16"), (lambda a: a.shared(q=a.heads(heads=3)), "multiple"),
    (lambda a: a.shared(scale=math.inf), "scale"), (lambda a: a.shared(scores=a.form(math.nan)), "cap"),
    (lambda a: a.shared(out=a.heads(type=1)), "out"), (lambda a: a.shared(lse=a.p + 1), "lse"),
    (lambda a: a.shared(ws=a.p + 16), "workspace"), (lambda a: a.shared(n=16384), "workspace"),
    (lambda a: a.shared(seqs=a.seqs(table_width=1 << 28, table_stride=1 << 28),
                        prefix=a.seqs(table_width=1 << 28, table_stride=1 << 28)), "2^31"),
]


@pytest.mark.parametrize("i", range(len(ABI_REFUSALS)))
def test_the_c_abi_refuses_before_any_cuda_call(E, i):
    a = Abi2(E)
    call, words = ABI_REFUSALS[i]
    assert call(a) == -1
    said = a.L.engram_last_error().decode()
    assert words in said and said.startswith("engram_"), said


def test_no_tokens_is_no_work(E):
    a = Abi2(E)
    none, nobody = a.heads(data=0), a.seqs(batch=0, block_table=None, seq_lens=None)
    assert a.prompt(T=0, q=none, out=none) == 0
    assert a.prompt(seqs=nobody, cu=None) == 0
    assert a.shared(seqs=nobody, q=none, out=none) == 0


def test_workspaces_grow_with_what_they_serve_and_refuse_bad_sizes(E):
    a = Abi2(E)
    c = C.byref(a.cache())
    p = [a.L.engram_prompt_workspace_bytes(c, 4, T, B) for T, B in ((0, 0), (1, 1), (100000, 1), (100000, 1000))]
    assert 16384 < p[0] <= p[1] < p[2] < p[3] and all(x % 256 == 0 for x in p)
    s = [a.L.engram_shared_workspace_bytes(c, 4, B, n) for B, n in ((0, 0), (1, 1), (1000, 1), (1000, 500))]
    assert s[0] < s[1] < s[2] <= s[3] and s[2] - s[1] >= 999 * 4 * 65 * 4
    for bad in ((None, 4, 1, 1), (c, 3, 1, 1), (c, 0, 1, 1), (c, 4, -1, 1), (c, 4, 1 << 31, 1), (c, 4, 1 << 30, 1), (c, 4, 1, -1)):
        assert a.L.engram_prompt_workspace_bytes(*bad) == 0
    for bad in ((None, 4, 1, 1), (c, 3, 1, 1), (c, 4, -1, 1), (c, 4, 1, -1), (c, 4, 1 << 30, 1)):
        assert a.L.engram_shared_workspace_bytes(*bad) == 0


# -------------------------------------------------------------------------------- pins of the oracle

def test_what_tokens_see():
    def seen(*args, **kw):
        p, lo, hi = A.visible(*args, **kw)
        return list(zip(p.tolist(), lo.tolist(), hi.tolist()))

    assert seen(2, 5) == [(3, 0, 4), (4, 0, 5)]
    assert seen(2, 5, causal=False) == [(3, 0, 5), (4, 0, 5)]
    assert seen(3, 5, window=2) == [(2, 1, 3), (3, 2, 4), (4, 3, 5)]
    assert seen(3, 3, doc_starts=np.array([0, 1, 1])) == [(0, 0, 1), (1, 1, 2), (2, 1, 3)]
    assert seen(3, 3, prefix_ends=np.array([2, 2, 9])) == [(0, 0, 2), (1, 0, 2), (2, 0, 3)]
    # more new tokens than the length holds: the first one stands before position 0 and sees nothing
    p, lo, hi = A.visible(3, 2)
    assert p.tolist() == [-1, 0, 1] and hi.tolist() == [0, 1, 2]


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (2.0, 0.0), (0.0, 0.5), (2.0, 0.5)])
def test_oracle_rows_against_a_sum_written_out(cap, slope):
    rng = np.random.default_rng(5)
    T, n, Hq, Hk, D = 4, 6, 4, 2, 8
    q, k, v = rng.standard_normal((T, Hq, D)), rng.standard_normal((n, Hk, D)), rng.standard_normal((n, Hk, D))
    p, lo, hi = A.visible(T, n, window=3)
    seen = (np.arange(n) >= lo[:, None]) & (np.arange(n) < hi[:, None])
    seen[1] = False
    out, lse, tol, tol_lse = A.attention_rows(q, k, v, seen, p, 0.3, cap, np.full(Hq, slope) if slope else None)
    for t in range(T):
        for h in range(Hq):
            total, o = 0.0, np.zeros(D)
            for j in range(n):
                if seen[t, j]:
                    x = 0.3 * float(q[t, h] @ k[j, h // 2])
                    w = math.exp((cap * math.tanh(x / cap) if cap else x) - slope * abs(int(p[t]) - j))
                    total, o = total + w, o + w * v[j, h // 2]
            if total == 0.0:
                assert not out[t, h].any() and lse[t, h] == -np.inf
            else:
                np.testing.assert_allclose(out[t, h], o / total, rtol=1e-12, atol=1e-12)
                assert abs(lse[t, h] - math.log(total)) < 1e-12
                assert (tol[t, h] > 0).all() and tol_lse[t, h] > 0
