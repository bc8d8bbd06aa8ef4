"""The attention operators without a GPU: their refusals (shapes and types in the binding, pointers, strides
and sizes in the C ABI, each before any CUDA call) and the pins of their 64-bit oracle."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import attention_oracle as A


@pytest.fixture(scope="module")
def E():
    from engram_gram_hash_02_gb300 import build as B
    B.build()
    import engram_gram_hash_02_gb300 as E
    return E


# ------------------------------------------------------------------------------------- the binding

B_, HQ, HK, D, PAGE, PAGES = 3, 4, 2, 64, 16, 10


def _good(E, fmt="bf16"):
    cache = E.KVCache.allocate(PAGES, PAGE, HK, D, fmt, device="cpu")
    w = torch.ones(D, dtype=torch.bfloat16)
    nr = E.NormRope(w, w, 1e-6, E.rope_table(32, D, device="cpu"))
    rows = {h: torch.zeros(B_, n, D, dtype=torch.bfloat16) for h, n in (("q", HQ), ("k", HK), ("v", HK))}
    return dict(cache=cache, nr=nr, **rows, positions=torch.zeros(B_, dtype=torch.int32), slots=torch.zeros(B_, dtype=torch.int64),
                block_table=torch.zeros(B_, 4, dtype=torch.int32), seq_lens=torch.ones(B_, dtype=torch.int32))


CALLS = {
    "engram_qk_norm_rope": ("nr", "q", "k", "positions"),
    "engram_kv_write": ("cache", "k", "v", "slots"),
    "engram_kv_read": ("cache", "slots"),
    "engram_paged_attention": ("cache", "q", "block_table", "seq_lens"),
    "engram_attention_step": ("nr", "cache", "q", "k", "v", "positions", "slots", "block_table", "seq_lens"),
}


def _call(E, fn, a, **more):
    return getattr(E, fn)(*(a[n] for n in CALLS[fn]), **more)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("fn", sorted(CALLS))
def test_well_formed_cpu_tensors_are_refused_for_their_device_only(E, fn, fmt):
    with pytest.raises(ValueError, match="CUDA"):
        _call(E, fn, _good(E, fmt))


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


REFUSALS = [
    # call, what is replaced, by what, words of the message
    ("engram_qk_norm_rope", "q", lambda: _z(B_, HQ, D, 1), "dimensions"),
    ("engram_qk_norm_rope", "q", lambda: _z(B_, HQ, D, dtype=torch.float16), "bfloat16"),
    ("engram_qk_norm_rope", "k", lambda: _z(B_ + 1, HK, D), "k must have shape"),
    ("engram_qk_norm_rope", "k", lambda: _z(B_, HK, 2 * D), "k must have shape"),
    ("engram_qk_norm_rope", "k", lambda: _z(B_, HK, D, dtype=torch.float32), "k must be"),
    ("engram_qk_norm_rope", "q", lambda: _z(B_, D, HQ).transpose(1, 2), "contiguous"),
    ("engram_qk_norm_rope", "positions", lambda: _z(B_, dtype=torch.int64), "positions"),
    ("engram_qk_norm_rope", "positions", lambda: _z(B_ + 1, dtype=torch.int32), "positions"),
    ("engram_qk_norm_rope", "positions", lambda: None, "positions"),
    ("engram_kv_write", "k", lambda: _z(B_, HQ, D), "k must have shape"),
    ("engram_kv_write", "v", lambda: _z(B_, HK, D + 1), "v must have shape"),
    ("engram_kv_write", "v", lambda: _z(B_, HK, D, dtype=torch.float32), "v must be"),
    ("engram_kv_write", "slots", lambda: _z(B_, dtype=torch.int32), "slots"),
    ("engram_kv_write", "slots", lambda: _z(2 * B_, dtype=torch.int64)[::2], "contiguous"),
    ("engram_kv_read", "slots", lambda: _z(B_, 1, dtype=torch.int64), "dimensions"),
    ("engram_kv_read", "slots", lambda: _z(B_, dtype=torch.int32), "slots"),
    ("engram_paged_attention", "q", lambda: _z(B_, HQ, D // 2), "heads of"),
    ("engram_paged_attention", "q", lambda: _z(B_, HK + 1, D), "multiple"),
    ("engram_paged_attention", "block_table", lambda: _z(B_ + 1, 4, dtype=torch.int32), "block_table"),
    ("engram_paged_attention", "block_table", lambda: _z(B_, 4, dtype=torch.int64), "block_table"),
    ("engram_paged_attention", "block_table", lambda: _z(4, B_, dtype=torch.int32).T, "contiguous"),
    ("engram_paged_attention", "seq_lens", lambda: _z(B_ - 1, dtype=torch.int32), "seq_lens"),
    ("engram_paged_attention", "seq_lens", lambda: _z(B_, dtype=torch.int64), "seq_lens"),
    ("engram_attention_step", "k", lambda: _z(B_, HQ, D), "k must have shape"),
    ("engram_attention_step", "v", lambda: _z(B_, HK, D, dtype=torch.float32), "v must be"),
    ("engram_attention_step", "positions", lambda: None, "positions"),
    ("engram_attention_step", "slots", lambda: _z(B_ + 1, dtype=torch.int64), "slots"),
]


@pytest.mark.parametrize("fn,name,make,words", REFUSALS)
def test_the_binding_refuses(E, fn, name, make, words):
    a = _good(E)
    a[name] = make()
    with pytest.raises((ValueError, TypeError), match=words):
        _call(E, fn, a)


@pytest.mark.parametrize("fn,more,words", [
    ("engram_qk_norm_rope", dict(q_out=_z(B_, HQ + 1, D)), "q_out"),
    ("engram_qk_norm_rope", dict(k_out=_z(B_, HK, D, dtype=torch.float16)), "k_out"),
    ("engram_kv_read", dict(k_out=_z(B_, HK, D + 2)), "k_out"),
    ("engram_paged_attention", dict(out=_z(B_, HQ, D, dtype=torch.float32)), "out"),
    ("engram_paged_attention", dict(lse=_z(B_, HQ)), "lse"),
    ("engram_paged_attention", dict(lse=3), "lse"),
    ("engram_paged_attention", dict(window=-1), "window"),
    ("engram_paged_attention", dict(workspace=_z(64)), "workspace"),
    ("engram_paged_attention", dict(err=_z(1)), "err"),
])
def test_the_binding_refuses_outputs_and_options(E, fn, more, words):
    with pytest.raises((ValueError, TypeError), match=words):
        _call(E, fn, _good(E), **more)


def test_what_a_program_keeps_is_checked_when_it_is_made(E):
    w = torch.ones(D, dtype=torch.bfloat16)
    for bad in (lambda: E.NormRope(w, None, 1e-6, None), lambda: E.NormRope(w.float(), w.float(), 1e-6, None),
                lambda: E.NormRope(w, w, 1e-6, torch.zeros(4, 8, dtype=torch.float64)), lambda: E.rope_table(4, 7),
                lambda: E.KVCache(_z(2, 2, 8, 64), _z(2, 2, 8, 32)), lambda: E.KVCache(_z(2, 2, 64), _z(2, 2, 64)),
                lambda: E.KVCache(_z(2, 2, 8, 64), _z(2, 8, 2, 64).transpose(1, 2)),
                lambda: E.KVCache(_z(2, 2, 8, 64, dtype=torch.uint8), _z(2, 2, 8, 64, dtype=torch.uint8)),
                lambda: E.KVCache(_z(2, 2, 8, 64), _z(2, 2, 8, 64), _z(2, 2, 8, 4, dtype=torch.uint8), _z(2, 2, 8, 4, dtype=torch.uint8)),
                lambda: E.KVCache.allocate(2, 8, 2, 64, "int8", device="cpu")):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(ValueError, match="q_weight"):
        E.engram_qk_norm_rope(E.NormRope(w[:32].clone(), w[:32].clone(), 1e-6, None), _z(2, 2, D), None, None)
    cache = E.KVCache.allocate(2, 8, 2, 160, "fp8", device="cpu")
    assert cache.k_scales.shape == (2, 2, 8, 8) and cache.fmt == "fp8"
    with pytest.raises(ValueError):
        E.attention_workspace(cache, 3, 1)
    assert E.attention_workspace_bytes(cache, 4, 8) % 256 == 0
    assert not E.attention_workspace(cache, 4, 8)[:16384].any()


# --------------------------------------------------------------------------------------- the C ABI

class Abi:
    """Well-formed arguments of the five calls on host memory (a check that fails launches nothing)."""

    def __init__(self, E):
        from engram_gram_hash_02_gb300 import attention as M, binding
        self.M, self.L = M, binding.lib()
        self.buf = (C.c_uint8 * 8192)()
        self.p = (C.addressof(self.buf) + 255) & ~255

    def heads(self, heads=2, ts=128, hs=64, type=0, data=None):
        return self.M._Heads(self.p if data is None else data, ts, hs, heads, type)

    def cache(self, **kw):
        c = self.M._Cache(1, 2, 64, 8, 4, self.p, self.p, 1024, 512, 64, self.p, self.p, 64, 32, 4)
        for n, x in kw.items():
            setattr(c, n, x)
        return c

    def nr(self, **kw):
        r = self.M._NormRope(self.p, self.p, 1e-6, self.p, 8, 64, 0, 0)
        for n, x in kw.items():
            setattr(r, n, x)
        return r

    def seqs(self, **kw):
        s = self.M._Seqs(2, self.p, 4, 4, self.p)
        for n, x in kw.items():
            setattr(s, n, x)
        return s

    def norm(self, nr=None, T=2, D=64, q=None, k=None, pos=True, qo=None, ko=None):
        r = [None if x is False else C.byref(x or self.heads()) for x in (q, k, qo, ko)]
        return self.L.engram_qk_norm_rope(C.byref(nr or self.nr()), T, D, r[0], r[1], self.p if pos else None, r[2], r[3], None, None)

    def write(self, cache=None, T=2, k=None, v=None, slots=True):
        return self.L.engram_kv_write(C.byref(cache or self.cache()), T, C.byref(k or self.heads()), C.byref(v or self.heads()),
                                      self.p if slots is True else slots, None, None)

    def read(self, cache=None, T=2, k=None, v=None, slots=True):
        return self.L.engram_kv_read(C.byref(cache or self.cache()), T, self.p if slots is True else slots,
                                     C.byref(k or self.heads()), C.byref(v or self.heads()), None, None)

    def attend(self, cache=None, seqs=None, q=None, scale=0.1, window=0, out=None, lse=None, ws=True, n=1 << 40):
        return self.L.engram_paged_attention(C.byref(cache or self.cache()), C.byref(seqs or self.seqs()),
                                             C.byref(q or self.heads()), scale, window, C.byref(out or self.heads()), lse,
                                             self.p if ws is True else ws, n, None, None)

    def step(self, nr=None, cache=None, seqs=None, q=None, k=None, v=None, pos=True, slots=True, out=None, n=1 << 40):
        h = [C.byref(x or self.heads()) for x in (q, k, v)]
        return self.L.engram_attention_step(C.byref(nr or self.nr()), C.byref(cache or self.cache()), C.byref(seqs or self.seqs()), *h,
                                            self.p if pos else None, self.p if slots else None, 0.1, 0,
                                            C.byref(out or self.heads()), None, self.p, n, None, None)


ABI_REFUSALS = [
    (lambda a: a.norm(D=60), "head_dim"), (lambda a: a.norm(D=264), "head_dim"), (lambda a: a.norm(T=-1), "T must"),
    (lambda a: a.norm(q=False, qo=False, k=False, ko=False), "q with q_out"), (lambda a: a.norm(q=False), "q with q_out"),
    (lambda a: a.norm(nr=a.nr(k_weight=None)), "both"), (lambda a: a.norm(nr=a.nr(q_weight=a.p + 2)), "aligned"),
    (lambda a: a.norm(nr=a.nr(eps=-1.0)), "eps"), (lambda a: a.norm(nr=a.nr(eps=math.nan)), "eps"),
    (lambda a: a.norm(nr=a.nr(rope_dim=72)), "rotated part"), (lambda a: a.norm(nr=a.nr(rope_dim=48, rope_start=24)), "rotated part"),
    (lambda a: a.norm(nr=a.nr(rope_dim=24)), "rope_dim"), (lambda a: a.norm(nr=a.nr(rope_dim=32, rope_start=4)), "rope_start"),
    (lambda a: a.norm(nr=a.nr(table=None)), "table"), (lambda a: a.norm(nr=a.nr(table_rows=0)), "row"),
    (lambda a: a.norm(pos=False), "positions"), (lambda a: a.norm(q=a.heads(data=a.p + 8)), "16 bytes"),
    (lambda a: a.norm(q=a.heads(ts=132)), "16 bytes"), (lambda a: a.norm(k=a.heads(hs=68)), "16 bytes"),
    (lambda a: a.norm(q=a.heads(type=2)), "type"), (lambda a: a.norm(q=a.heads(heads=0)), "heads"),
    (lambda a: a.norm(q=a.heads(ts=-128)), "strides"), (lambda a: a.norm(qo=a.heads(ts=64)), "overlap"),
    (lambda a: a.norm(qo=a.heads(hs=32)), "overlap"), (lambda a: a.norm(qo=a.heads(heads=1)), "q_out"),
    (lambda a: a.norm(k=a.heads(type=1)), "one type"),
    (lambda a: a.write(cache=a.cache(format=2)), "format"), (lambda a: a.write(cache=a.cache(head_dim=48)), "head_dim"),
    (lambda a: a.write(cache=a.cache(format=0, head_dim=24)), "head_dim"), (lambda a: a.write(cache=a.cache(head_dim=288)), "head_dim"),
    (lambda a: a.write(cache=a.cache(page_size=0)), "page_size"), (lambda a: a.write(cache=a.cache(num_pages=-1)), "num_pages"),
    (lambda a: a.write(cache=a.cache(kv_heads=0)), "kv_heads"), (lambda a: a.write(cache=a.cache(k=None)), "non-NULL"),
    (lambda a: a.write(cache=a.cache(v=a.p + 4)), "aligned"), (lambda a: a.write(cache=a.cache(token_stride=72)), "16 bytes"),
    (lambda a: a.write(cache=a.cache(head_stride=-64)), ">= 0"), (lambda a: a.write(cache=a.cache(k_scales=None)), "scales"),
    (lambda a: a.write(cache=a.cache(scale_token_stride=2)), "scale strides"), (lambda a: a.write(k=a.heads(heads=3)), "heads"),
    (lambda a: a.write(v=a.heads(type=1)), "one type"), (lambda a: a.write(slots=None), "slots"),
    (lambda a: a.write(slots=a.p + 4), "slots"), (lambda a: a.write(T=1 << 31), "T must"),
    (lambda a: a.read(slots=None), "slots"), (lambda a: a.read(k=a.heads(ts=0)), "overlap"),
    (lambda a: a.read(v=a.heads(heads=1)), "heads"),
    (lambda a: a.attend(q=a.heads(heads=3)), "multiple"), (lambda a: a.attend(seqs=a.seqs(batch=-1)), "batch"),
    (lambda a: a.attend(seqs=a.seqs(table_stride=3)), "stride"), (lambda a: a.attend(seqs=a.seqs(block_table=None)), "block_table"),
    (lambda a: a.attend(seqs=a.seqs(seq_lens=None)), "seq_lens"), (lambda a: a.attend(scale=math.inf), "scale"),
    (lambda a: a.attend(scale=math.nan), "scale"), (lambda a: a.attend(window=-2), "window"),
    (lambda a: a.attend(out=a.heads(type=1)), "out"), (lambda a: a.attend(out=a.heads(heads=4, hs=64, ts=256)), "out"),
    (lambda a: a.attend(out=a.heads(ts=64)), "overlap"), (lambda a: a.attend(lse=a.p + 2), "lse"),
    (lambda a: a.attend(ws=None), "workspace"), (lambda a: a.attend(ws=a.p + 128), "workspace"),
    (lambda a: a.attend(n=4096), "workspace"),
    (lambda a: a.attend(seqs=a.seqs(batch=1 << 30, table_width=1 << 20, table_stride=1 << 20)), "too large"),
    (lambda a: a.step(k=a.heads(heads=4, ts=256)), "heads"), (lambda a: a.step(q=a.heads(type=1)), "one type"),
    (lambda a: a.step(q=a.heads(heads=3)), "multiple"), (lambda a: a.step(pos=False), "positions"),
    (lambda a: a.step(slots=False), "slots"), (lambda a: a.step(nr=a.nr(rope_dim=128)), "rotated part"),
    (lambda a: a.step(n=4096), "workspace"),
]


@pytest.mark.parametrize("i", range(len(ABI_REFUSALS)))
def test_the_c_abi_refuses_before_any_cuda_call(E, i):
    a = Abi(E)
    call, words = ABI_REFUSALS[i]
    assert call(a) == -1
    said = a.L.engram_last_error().decode()
    assert words in said and said.startswith("engram_"), said


def test_no_tokens_is_no_work(E):
    a = Abi(E)
    none = a.heads()
    none.data = None
    assert a.norm(T=0, q=none, qo=none, k=none, ko=none, pos=False) == 0
    assert a.write(T=0, k=none, v=none, slots=None) == 0 and a.read(T=0, k=none, v=none, slots=None) == 0
    nobody = a.seqs(batch=0, block_table=None, seq_lens=None)
    assert a.attend(seqs=nobody, q=none, out=none) == 0
    assert a.step(seqs=nobody, q=none, k=none, v=none, out=none, pos=False, slots=False) == 0


def test_workspace_covers_the_join_and_the_turned_queries(E):
    a = Abi(E)
    small, big = (a.L.engram_attention_workspace_bytes(C.byref(a.cache()), 4, b) for b in (1, 1000))
    assert big - small >= 999 * 4 * 64 * 4 and small > 16384
    assert a.L.engram_attention_workspace_bytes(C.byref(a.cache()), 3, 1) == 0
    assert a.L.engram_attention_workspace_bytes(None, 4, 1) == 0


# -------------------------------------------------------------------------------- pins of the oracle

def test_oracle_rotation_keeps_norms_and_composes():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(6, 3, 32))
    t = A.rope_angles(20, 16)
    for inter in (False, True):
        y = A.norm_rope(x, None, 0.0, t, np.arange(6), 8, inter)
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-6)
        assert np.array_equal(y[..., :8], x[..., :8]) and np.array_equal(y[..., 24:], x[..., 24:])
        assert np.allclose(A.norm_rope(x, None, 0.0, t, np.zeros(6, int), 8, inter), x, atol=1e-12)
        # the product of two rows depends on the distance of their positions only
        a, b = (A.norm_rope(x[:1], None, 0.0, t, [p], 8, inter) for p in (3, 10))
        c, d = (A.norm_rope(x[1:2], None, 0.0, t, [p], 8, inter) for p in (5, 12))
        assert np.allclose((a * c).sum(-1), (b * d).sum(-1), rtol=1e-5, atol=1e-5)
    by_hand = A.norm_rope(np.array([[[3.0, 4.0]]]), np.array([1.0, 2.0]), 0.0, np.array([[0.0, 1.0]]), [0])
    n = math.sqrt(12.5)
    assert np.allclose(by_hand, [[[-8.0 / n, 3.0 / n]]])


def test_oracle_codes_are_torchs_casts_and_scales_are_smallest():
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(200, 2, 64)) * np.exp2(30 * rng.normal(size=(200, 2, 1)))).astype(np.float32)
    x = np.clip(x, -3e38, 3e38)
    codes, bytes_ = A.fp8_encode(x)
    scale = np.repeat(np.exp2(bytes_.astype(np.float64) - 127), 32, -1)
    cast = torch.from_numpy(x / scale).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, cast)
    top = np.abs(x.astype(np.float64)).reshape(200, 2, 2, 32).max(-1) / np.exp2(bytes_.astype(np.float64) - 127)
    assert (top <= 448).all() and ((top > 224) | (bytes_ == 1)).all()
    every = np.concatenate([np.arange(127), 128 + np.arange(127)]).astype(np.uint8)
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    pad = np.concatenate([every, np.zeros(2, np.uint8)])
    assert np.array_equal(A.fp8_decode(pad, np.full(8, 127, np.uint8))[:254], want)


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(9, 2, 16)), rng.normal(size=(9, 2, 16))
    q = rng.normal(size=(6, 16))
    out, lse, _, _ = A.attention(q, k, v, 0.0)
    assert np.allclose(out[:3], v[:, 0].mean(0)) and np.allclose(out[3:], v[:, 1].mean(0)) and np.allclose(lse, math.log(9))
    out, lse, _, _ = A.attention(q, k[:1], v[:1], 0.7)
    assert np.allclose(out[0], v[0, 0]) and np.allclose(lse[5], 0.7 * q[5] @ k[0, 1])
    out, lse, _, _ = A.attention(q, k[:0], v[:0], 1.0)
    assert not out.any() and np.all(lse == -np.inf)
    t = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q)[:, None], torch.from_numpy(k).transpose(0, 1).repeat_interleave(3, 0),
        torch.from_numpy(v).transpose(0, 1).repeat_interleave(3, 0))
    assert np.allclose(A.attention(q, k, v, 0.25)[0], t[:, 0].numpy())
