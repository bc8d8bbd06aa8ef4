"""ctypes binding of libengram's attention calls: argument marshalling only.

The layer's attention next to its Engram residual: per-head norms of queries and keys with the
position rotation, rows written to a paged key-value cache (bf16, or e4m3 codes with one scale byte
per 32 values) and read back, attention of one new token per sequence over the cache, and all of
them as one decode step; attention of all tokens of prompts (causal, with a window, documents or a
prefix seen both ways), and of batches whose sequences share a prefix. Scores may be capped by a tanh
(``cap``) and carry a bias that falls with distance (``slopes``).

Every call has two forms, as ``engram_forward`` has: a function that checks, runs and returns its
outputs, and a plan (``...Plan``) that marshals the call once for fixed tensors and runs it with one
ctypes call (``plan.run(stream)``; the outputs are its attributes). Tensors may be strided views as
long as a head's values are contiguous. Outputs that are not given are allocated for the stream the
call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes as C

import torch

from .binding import _check, _ptr, _shape, _stream, lib

CACHE_BF16, CACHE_FP8_E8M0 = 0, 1
ATTENTION_ZERO_BYTES = 16384   # ENGRAM_ATTENTION_ZERO_BYTES
_TYPES = {torch.bfloat16: 0, torch.float32: 1}


class _Heads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64), ("heads", C.c_int32),
                ("type", C.c_int32)]


class _Cache(C.Structure):
    _fields_ = [("format", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("page_size", C.c_int32),
                ("num_pages", C.c_int64), ("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64),
                ("head_stride", C.c_int64), ("token_stride", C.c_int64), ("k_scales", C.c_void_p),
                ("v_scales", C.c_void_p), ("scale_page_stride", C.c_int64), ("scale_head_stride", C.c_int64),
                ("scale_token_stride", C.c_int64)]


class _NormRope(C.Structure):
    _fields_ = [("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("eps", C.c_float), ("table", C.c_void_p),
                ("table_rows", C.c_int64), ("rope_dim", C.c_int32), ("rope_start", C.c_int32),
                ("interleaved", C.c_int32)]


class _Seqs(C.Structure):
    _fields_ = [("batch", C.c_int32), ("block_table", C.c_void_p), ("table_stride", C.c_int64),
                ("table_width", C.c_int32), ("seq_lens", C.c_void_p)]


class _Scores(C.Structure):
    _fields_ = [("cap", C.c_float), ("slopes", C.c_void_p)]


class _Visible(C.Structure):
    _fields_ = [("causal", C.c_int32), ("window", C.c_int32), ("doc_starts", C.c_void_p), ("prefix_ends", C.c_void_p)]


# ---------------------------------------------------------------------------------------------
# checks (shapes first, so that they can be reached without a GPU)
# ---------------------------------------------------------------------------------------------

def _tensor(t, dim: int, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions (got shape {tuple(t.shape)})")
    return t


def _on(device, **tensors):
    """Every tensor on one CUDA device: the kernels take raw pointers."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _typed(t, dtypes, name: str):
    if t is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")


def _rows(t, name: str, shape=None) -> torch.Tensor:
    """[T, heads, D] rows of bf16 or fp32 whose last axis is contiguous."""
    _tensor(t, 3, name)
    if shape is not None:
        _shape(t, shape, name)
    _typed(t, tuple(_TYPES), name)
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous heads (last stride 1)")
    return t


def _vector(t, n: int, dtype, name: str):
    if t is None:
        return
    _shape(t, (n,), name)
    _typed(t, (dtype,), name)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _strides(t, n: int):
    """The first n strides; an axis of one entry is never stepped along, whatever its stride says."""
    return tuple(0 if t.shape[i] <= 1 else t.stride(i) for i in range(n))


def _heads(t) -> _Heads:
    return _Heads(t.data_ptr(), *_strides(t, 2), t.shape[1], _TYPES[t.dtype])


def _err(err):
    if err is not None:
        if not isinstance(err, torch.Tensor) or err.dtype != torch.int32 or err.numel() < 1:
            raise ValueError("err must be an int32 tensor that holds one word")


def _alloc(shape, dtype, device, stream):
    """An output that belongs to the stream its call runs on (the caching allocator hands memory on in
    the order of the stream it was taken for)."""
    with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
        return torch.empty(shape, dtype=dtype, device=device)


# a plan's run() is a few microseconds of host time: the current stream as a number, without an object for it
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class _Plan:
    """A call of the library marshalled once for fixed tensors. The tensors are kept alive; run() enqueues
    the call on `stream` (default: the current stream of the plan's device).

    What the plan made itself (`made`: outputs, a workspace and its zeros) belongs to the stream it was made
    on: `home`. The first run on any other stream waits for what has been enqueued there, and the memory goes
    back only when that stream is done with it, too. Nothing of this enters a graph: a run that is captured on
    a stream of its own is the caller's to order after the plan's making (torch.cuda.graph synchronises)."""

    def __init__(self, fn: str, device, keep, *args, made=(), home=None):
        self._name, self._fn, self._args, self._keep, self._device = fn, getattr(lib(), fn), args, keep, device
        self._made = tuple(t for t in made if t is not None)
        if self._made:
            self._home = torch.cuda.current_stream(device) if home is None else home
            self._ordered = {self._home.cuda_stream}

    def _order(self, stream):
        if _capturing(stream) or _capturing(self._home):
            return
        stream.wait_stream(self._home)
        for t in self._made:
            t.record_stream(stream)
        self._ordered.add(stream.cuda_stream)

    def run(self, stream=None):
        index = self._device.index
        s = _current_raw_stream(index) if stream is None else stream.cuda_stream
        if self._made and s not in self._ordered:
            self._order(torch.cuda.current_stream(self._device) if stream is None else stream)
        if _current_device() == index:
            rc = self._fn(*self._args, s)
        else:
            with torch.cuda.device(self._device):
                rc = self._fn(*self._args, s)
        if rc != 0:
            _check(self._name, rc)


# ---------------------------------------------------------------------------------------------
# what a program keeps
# ---------------------------------------------------------------------------------------------

def rope_table(positions: int, rope_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation table fp32 [positions, rope_dim] (cosines, then sines) of the angles
    p * base^(-2i / rope_dim), computed in 64 bits (host setup, once per model)."""
    if rope_dim < 2 or rope_dim % 2:
        raise ValueError(f"rope_dim must be even and >= 2 (got {rope_dim})")
    inv = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


class NormRope:
    """The norm and rotation of a layer's queries and keys (EngramNormRope): weights bf16 [D] (both, or
    None for no norm) and a table fp32 [positions, rope_dim] (None for no rotation; see ``rope_table``).
    The rotation turns values [start, start + rope_dim) of a head, in halves or (interleaved) in pairs."""

    def __init__(self, q_weight, k_weight, eps: float, table, start: int = 0, interleaved: bool = False):
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight must both be given, or neither")
        for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _tensor(t, 1, n)
                _typed(t, (torch.bfloat16,), n)
                if not t.is_contiguous():
                    raise ValueError(f"{n} must be contiguous")
        if table is not None:
            _tensor(table, 2, "table")
            _typed(table, (torch.float32,), "table")
            if not table.is_contiguous():
                raise ValueError("table must be contiguous")
        self.q_weight, self.k_weight, self.table = q_weight, k_weight, table
        self._c = _NormRope(_ptr(q_weight), _ptr(k_weight), float(eps), _ptr(table), 0 if table is None else table.shape[0],
                            0 if table is None else table.shape[1], int(start), 1 if interleaved else 0)

    def _fits(self, D: int):
        for t, n in ((self.q_weight, "q_weight"), (self.k_weight, "k_weight")):
            _shape(t, (D,), n)


class KVCache:
    """A paged cache of keys and values (EngramKVCache): k and v [pages, kv_heads, page_size, head_dim]
    of equal strides, any views whose last axis is contiguous (a [pages, page_size, kv_heads, head_dim]
    buffer enters as its ``transpose(1, 2)``). bf16, or e4m3 codes (uint8) with k_scales and v_scales,
    uint8 [pages, kv_heads, page_size, 4 * ceil(head_dim / 128)]: byte b is the scale of values
    32b .. 32b + 31. Slot s is place s % page_size of page s // page_size."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        _tensor(k, 4, "k")
        _tensor(v, 4, "v")
        _shape(v, k.shape, "v")
        _typed(k, (torch.bfloat16, torch.uint8), "k")
        _typed(v, (k.dtype,), "v")
        fp8 = k.dtype == torch.uint8
        if _strides(k, 4) != _strides(v, 4) or (k.shape[3] > 1 and k.stride(3) != 1):
            raise ValueError("k and v must have equal strides and contiguous heads (last stride 1)")
        s = (0, 0, 0)
        if fp8:
            if k_scales is None or v_scales is None:
                raise ValueError("an FP8 cache needs k_scales and v_scales")
            for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
                _shape(t, (*k.shape[:3], 4 * -(-k.shape[3] // 128)), n)
                _typed(t, (torch.uint8,), n)
                if t.stride(3) != 1:
                    raise ValueError(f"{n} must have contiguous words (last stride 1)")
            if _strides(k_scales, 3) != _strides(v_scales, 3):
                raise ValueError("k_scales and v_scales must have equal strides")
            s = _strides(k_scales, 3)
        elif k_scales is not None or v_scales is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self._c = _Cache(CACHE_FP8_E8M0 if fp8 else CACHE_BF16, self.kv_heads, self.head_dim, self.page_size,
                         self.num_pages, k.data_ptr(), v.data_ptr(), *_strides(k, 3), _ptr(k_scales), _ptr(v_scales), *s)

    @property
    def fmt(self) -> str:
        return "fp8" if self.k.dtype == torch.uint8 else "bf16"

    @property
    def device(self):
        return self.k.device

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: str = "bf16", device="cuda"):
        """A cache with the tokens of a page and head next to each other (an attention reads them in runs)."""
        if fmt not in ("bf16", "fp8"):
            raise ValueError(f"unknown cache format {fmt!r}")
        shape = (num_pages, kv_heads, page_size, head_dim)
        dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
        k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        if fmt == "bf16":
            return cls(k, v)
        words = (*shape[:3], 4 * -(-head_dim // 128))
        return cls(k, v, *(torch.full(words, 127, dtype=torch.uint8, device=device) for _ in range(2)))

    def _on(self, device):
        _on(device, **{"cache.k": self.k, "cache.v": self.v, "cache.k_scales": self.k_scales, "cache.v_scales": self.v_scales})


def attention_workspace_bytes(cache: KVCache, q_heads: int, batch: int) -> int:
    return int(lib().engram_attention_workspace_bytes(C.byref(cache._c), int(q_heads), int(batch)))


def _workspace(n: int, cache: KVCache, q_heads: int) -> torch.Tensor:
    if n == 0:
        raise ValueError(f"no workspace for {q_heads} query heads over {cache.kv_heads} key heads of {cache.head_dim}")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:ATTENTION_ZERO_BYTES].zero_()
    return ws


def attention_workspace(cache: KVCache, q_heads: int, batch: int) -> torch.Tensor:
    """A workspace of the attention calls on this cache for up to `batch` sequences. Its start
    (ATTENTION_ZERO_BYTES) is zero, and every call leaves it so: a program keeps one for calls that run in
    order. The zeros are written on the current stream; calls on another one are the caller's to order after it."""
    return _workspace(attention_workspace_bytes(cache, q_heads, batch), cache, q_heads)


def prompt_workspace_bytes(cache: KVCache, q_heads: int, tokens: int, batch: int) -> int:
    return int(lib().engram_prompt_workspace_bytes(C.byref(cache._c), int(q_heads), int(tokens), int(batch)))


def prompt_workspace(cache: KVCache, q_heads: int, tokens: int, batch: int) -> torch.Tensor:
    """A workspace of engram_prompt_attention on this cache for up to `tokens` new tokens of `batch` sequences; as
    ``attention_workspace``, and one that is large enough serves all the attention calls in order."""
    return _workspace(prompt_workspace_bytes(cache, q_heads, tokens, batch), cache, q_heads)


def shared_workspace_bytes(cache: KVCache, q_heads: int, batch: int, groups: int) -> int:
    return int(lib().engram_shared_workspace_bytes(C.byref(cache._c), int(q_heads), int(batch), int(groups)))


def shared_workspace(cache: KVCache, q_heads: int, batch: int, groups: int) -> torch.Tensor:
    """A workspace of engram_shared_attention on this cache for up to `batch` sequences in `groups` groups; as
    ``attention_workspace``."""
    return _workspace(shared_workspace_bytes(cache, q_heads, batch, groups), cache, q_heads)


# ---------------------------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------------------------

class QKNormRopePlan(_Plan):
    """engram_qk_norm_rope for fixed tensors: q [T, Hq, D] and k [T, Hk, D] (either may be None) of one
    type; q_out and k_out bf16 or fp32 (bf16 if not given; the inputs themselves are fine)."""

    def __init__(self, nr: NormRope, q, k, positions, q_out=None, k_out=None, err=None, stream=None):
        if q is None and k is None:
            raise ValueError("q, k or both must be given")
        lead = q if q is not None else k
        _rows(lead, "q" if q is not None else "k")
        T, _, D = lead.shape
        nr._fits(D)
        for t, o, n in ((q, q_out, "q"), (k, k_out, "k")):
            if t is None:
                if o is not None:
                    raise ValueError(f"{n}_out is given without {n}")
                continue
            _rows(t, n, (T, t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 3 else 1, D))
            _typed(t, (lead.dtype,), n)
            if o is not None:
                _rows(o, f"{n}_out", t.shape)
        if nr.table is not None and positions is None:
            raise ValueError("positions are needed with a rotation table")
        _vector(positions, T, torch.int32, "positions")
        _err(err)
        _on(lead.device, q=q, k=k, positions=positions, q_out=q_out, k_out=k_out, err=err, q_weight=nr.q_weight,
            k_weight=nr.k_weight, table=nr.table)
        made = []
        if q is not None and q_out is None:
            q_out = _alloc(q.shape, torch.bfloat16, q.device, stream)
            made.append(q_out)
        if k is not None and k_out is None:
            k_out = _alloc(k.shape, torch.bfloat16, k.device, stream)
            made.append(k_out)
        self.q_out, self.k_out = q_out, k_out
        ref = [None if t is None else C.byref(_heads(t)) for t in (q, k, q_out, k_out)]
        super().__init__("engram_qk_norm_rope", lead.device, (nr, q, k, positions, q_out, k_out, err), C.byref(nr._c), T, D,
                         ref[0], ref[1], _ptr(positions), ref[2], ref[3], _ptr(err), made=made, home=stream)


class KVWritePlan(_Plan):
    """engram_kv_write for fixed tensors: k and v [T, kv_heads, D] of one type to int64 slots [T], no two
    of them the same (below 0: skipped)."""

    def __init__(self, cache: KVCache, k, v, slots, err=None):
        _rows(k, "k")
        T = k.shape[0]
        _rows(k, "k", (T, cache.kv_heads, cache.head_dim))
        _rows(v, "v", k.shape)
        _typed(v, (k.dtype,), "v")
        _vector(slots, T, torch.int64, "slots")
        if slots is None:
            raise ValueError("slots must be given")
        _err(err)
        _on(k.device, k=k, v=v, slots=slots, err=err)
        cache._on(k.device)
        super().__init__("engram_kv_write", k.device, (cache, k, v, slots, err), C.byref(cache._c), T, C.byref(_heads(k)),
                         C.byref(_heads(v)), _ptr(slots), _ptr(err))


class KVReadPlan(_Plan):
    """engram_kv_read for fixed tensors: the rows at int64 slots [T] to k_out and v_out [T, kv_heads, D],
    bf16 or fp32 (bf16 if not given)."""

    def __init__(self, cache: KVCache, slots, k_out=None, v_out=None, err=None, stream=None):
        _tensor(slots, 1, "slots")
        T = slots.shape[0]
        _vector(slots, T, torch.int64, "slots")
        shape = (T, cache.kv_heads, cache.head_dim)
        for t, n in ((k_out, "k_out"), (v_out, "v_out")):
            if t is not None:
                _rows(t, n, shape)
        _err(err)
        _on(slots.device, slots=slots, k_out=k_out, v_out=v_out, err=err)
        cache._on(slots.device)
        made = []
        if k_out is None:
            k_out = _alloc(shape, torch.bfloat16, slots.device, stream)
            made.append(k_out)
        if v_out is None:
            v_out = _alloc(shape, k_out.dtype, slots.device, stream)
            made.append(v_out)
        self.k_out, self.v_out = k_out, v_out
        super().__init__("engram_kv_read", slots.device, (cache, slots, k_out, v_out, err), C.byref(cache._c), T, _ptr(slots),
                         C.byref(_heads(k_out)), C.byref(_heads(v_out)), _ptr(err), made=made, home=stream)


def _scores(cap, slopes, q_heads: int):
    """Checks of a form of scores: the EngramScores, or None without one."""
    cap = float(cap)
    if cap != 0.0 and not 2.0 ** -60 <= cap <= 2.0 ** 60:
        raise ValueError(f"cap must be 0 or in [2^-60, 2^60] (got {cap})")
    if slopes is not None:
        _tensor(slopes, 1, "slopes")
        _vector(slopes, q_heads, torch.float32, "slopes")
    return None if cap == 0.0 and slopes is None else _Scores(cap, _ptr(slopes))


def _paged_seqs(block_table, seq_lens, B: int, table: str = "block_table", lens: str = "seq_lens") -> _Seqs:
    """Checks of a page table and its lengths."""
    _tensor(block_table, 2, table)
    _shape(block_table, (B, block_table.shape[1]), table)
    _typed(block_table, (torch.int32,), table)
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError(f"{table} must have contiguous rows")
    _vector(seq_lens, B, torch.int32, lens)
    if seq_lens is None:
        raise ValueError(f"{lens} must be given")
    # a table of one row, or of one column, may have any stride there
    stride = max(block_table.stride(0), block_table.shape[1]) if B > 1 else block_table.shape[1]
    if B > 1 and block_table.stride(0) < block_table.shape[1]:
        raise ValueError(f"{table} rows overlap")
    return _Seqs(B, block_table.data_ptr(), stride, block_table.shape[1], seq_lens.data_ptr())


def _query(cache: KVCache, q, dtypes=tuple(_TYPES)):
    _rows(q, "q")
    _typed(q, dtypes, "q")
    if q.shape[2] != cache.head_dim:
        raise ValueError(f"q has heads of {q.shape[2]} but the cache of {cache.head_dim}")
    if q.shape[1] < 1 or q.shape[1] % cache.kv_heads:
        raise ValueError(f"q must have a multiple of the cache's {cache.kv_heads} heads (got {q.shape[1]})")
    return q.shape


def _attention_outputs(cache: KVCache, q, out, lse, workspace, err, stream, make_workspace, **others):
    """Checks and makes what an attention writes: (out, lse, workspace, what was made here). `others`: its other tensors."""
    T, Hq, _ = q.shape
    if out is not None:
        _rows(out, "out", q.shape)
        _typed(out, (torch.bfloat16,), "out")
    if isinstance(lse, torch.Tensor):
        _shape(lse, (T, Hq), "lse")
        _typed(lse, (torch.float32,), "lse")
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    elif lse is not None and not isinstance(lse, bool):
        raise TypeError("lse must be a tensor, or True to return one")
    if workspace is not None:
        _tensor(workspace, 1, "workspace")
        _typed(workspace, (torch.uint8,), "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _err(err)
    _on(q.device, q=q, out=out, lse=lse if isinstance(lse, torch.Tensor) else None, workspace=workspace, err=err, **others)
    cache._on(q.device)
    made = []
    if out is None:
        out = _alloc(q.shape, torch.bfloat16, q.device, stream)
        made.append(out)
    if lse is True:
        lse = _alloc((T, Hq), torch.float32, q.device, stream)
        made.append(lse)
    elif lse is False:
        lse = None
    if workspace is None:
        with torch.cuda.device(q.device), torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            workspace = make_workspace()
        made.append(workspace)
    return out, lse, workspace, made


def _scale(cache: KVCache, scale) -> float:
    return cache.head_dim ** -0.5 if scale is None else float(scale)


def _attention_args(cache: KVCache, q, block_table, seq_lens, scale, window, cap, slopes, out, lse, workspace, err, stream,
                    need_batch: int):
    """Checks and outputs of both one-token plans: (seqs, scale, window, scores, out, lse, workspace, what was made here)."""
    B, Hq, _ = _query(cache, q)
    seqs = _paged_seqs(block_table, seq_lens, B)
    if int(window) < 0:
        raise ValueError(f"window must be >= 0 (got {window})")
    scores = _scores(cap, slopes, Hq)
    out, lse, workspace, made = _attention_outputs(cache, q, out, lse, workspace, err, stream,
                                                   lambda: attention_workspace(cache, Hq, need_batch), block_table=block_table,
                                                   seq_lens=seq_lens, slopes=slopes)
    return seqs, _scale(cache, scale), int(window), scores, out, lse, workspace, made


class PagedAttentionPlan(_Plan):
    """engram_paged_attention for fixed tensors: q [B, Hq, D] (bf16 or fp32) over the cached tokens of B
    sequences (block_table int32 [B, width], seq_lens int32 [B]). scale defaults to D^-1/2; lse may be a
    tensor fp32 [B, Hq], or True to have one. Without a workspace the plan makes its own; plans that
    share one must run in order. With a cap (scores cap * tanh(s / cap)) or slopes (fp32 [Hq]: -slope per
    token of distance) it is engram_paged_attention2."""

    def __init__(self, cache: KVCache, q, block_table, seq_lens, scale=None, window: int = 0, out=None, lse=None, workspace=None,
                 err=None, stream=None, cap: float = 0.0, slopes=None):
        seqs, scale, window, scores, out, lse, workspace, made = _attention_args(cache, q, block_table, seq_lens, scale, window, cap,
                                                                                 slopes, out, lse, workspace, err, stream, 0)
        self.out, self.lse, self.workspace = out, lse, workspace
        fn, form = ("engram_paged_attention", ()) if scores is None else ("engram_paged_attention2", (C.byref(scores),))
        super().__init__(fn, q.device, (cache, q, block_table, seq_lens, slopes, out, lse, workspace, err), C.byref(cache._c),
                         C.byref(seqs), C.byref(_heads(q)), scale, window, *form, C.byref(_heads(out)), _ptr(lse), _ptr(workspace),
                         workspace.numel(), _ptr(err), made=made, home=stream)


class AttentionStepPlan(_Plan):
    """engram_attention_step for fixed tensors: the new tokens' q [B, Hq, D], k and v [B, Hk, D] (one
    type), positions int32 [B] and slots int64 [B]; the rest as PagedAttentionPlan."""

    def __init__(self, nr: NormRope, cache: KVCache, q, k, v, positions, slots, block_table, seq_lens, scale=None, window: int = 0,
                 out=None, lse=None, workspace=None, err=None, stream=None, cap: float = 0.0, slopes=None):
        _rows(q, "q")
        B, _, D = q.shape
        nr._fits(D)
        for t, n in ((k, "k"), (v, "v")):
            _rows(t, n, (B, cache.kv_heads, D))
            _typed(t, (q.dtype,), n)
        if nr.table is not None and positions is None:
            raise ValueError("positions are needed with a rotation table")
        _vector(positions, B, torch.int32, "positions")
        _vector(slots, B, torch.int64, "slots")
        if slots is None:
            raise ValueError("slots must be given")
        seqs, scale, window, scores, out, lse, workspace, made = _attention_args(cache, q, block_table, seq_lens, scale, window, cap,
                                                                                 slopes, out, lse, workspace, err, stream, B)
        _on(q.device, k=k, v=v, positions=positions, slots=slots, q_weight=nr.q_weight, k_weight=nr.k_weight, table=nr.table)
        self.out, self.lse, self.workspace = out, lse, workspace
        fn, form = ("engram_attention_step", ()) if scores is None else ("engram_attention_step2", (C.byref(scores),))
        super().__init__(fn, q.device,
                         (nr, cache, q, k, v, positions, slots, block_table, seq_lens, slopes, out, lse, workspace, err), C.byref(nr._c),
                         C.byref(cache._c), C.byref(seqs), C.byref(_heads(q)), C.byref(_heads(k)), C.byref(_heads(v)),
                         _ptr(positions), _ptr(slots), scale, window, *form, C.byref(_heads(out)), _ptr(lse), _ptr(workspace),
                         workspace.numel(), _ptr(err), made=made, home=stream)


class PromptAttentionPlan(_Plan):
    """engram_prompt_attention for fixed tensors: all new tokens q [T, Hq, D] (bf16) of B sequences, sequence b's the rows
    [cu_seqlens[b], cu_seqlens[b + 1]), over their cached tokens (block_table int32 [B, width], seq_lens int32 [B] with the
    new ones). New token i of n stands at position p = len - n + i and sees the keys [lo, hi): up to itself (causal), or up to
    prefix_ends[t] if that is further (int32 [T]); from doc_starts[t] on (int32 [T]), and at most `window` of them up to
    itself. out and lse keep what they hold in rows that belong to no sequence. The rest as PagedAttentionPlan."""

    def __init__(self, cache: KVCache, q, cu_seqlens, block_table, seq_lens, scale=None, causal: bool = True, window: int = 0,
                 doc_starts=None, prefix_ends=None, cap: float = 0.0, slopes=None, out=None, lse=None, workspace=None, err=None,
                 stream=None):
        T, Hq, _ = _query(cache, q, (torch.bfloat16,))
        _tensor(cu_seqlens, 1, "cu_seqlens")
        B = cu_seqlens.shape[0] - 1
        if B < 0:
            raise ValueError("cu_seqlens must have an entry for each sequence, and the end")
        _vector(cu_seqlens, B + 1, torch.int32, "cu_seqlens")
        seqs = _paged_seqs(block_table, seq_lens, B)
        if int(window) < 0:
            raise ValueError(f"window must be >= 0 (got {window})")
        _vector(doc_starts, T, torch.int32, "doc_starts")
        _vector(prefix_ends, T, torch.int32, "prefix_ends")
        if prefix_ends is not None and not causal:
            raise ValueError("prefix_ends are for causal attention")
        scores = _scores(cap, slopes, Hq)
        out, lse, workspace, made = _attention_outputs(cache, q, out, lse, workspace, err, stream,
                                                       lambda: prompt_workspace(cache, Hq, T, B), cu_seqlens=cu_seqlens,
                                                       block_table=block_table, seq_lens=seq_lens, doc_starts=doc_starts,
                                                       prefix_ends=prefix_ends, slopes=slopes)
        self.out, self.lse, self.workspace = out, lse, workspace
        visible = _Visible(1 if causal else 0, int(window), _ptr(doc_starts), _ptr(prefix_ends))
        super().__init__("engram_prompt_attention", q.device,
                         (cache, q, cu_seqlens, block_table, seq_lens, doc_starts, prefix_ends, slopes, out, lse, workspace, err),
                         C.byref(cache._c), C.byref(seqs), T, _ptr(cu_seqlens), C.byref(_heads(q)), _scale(cache, scale),
                         C.byref(visible), None if scores is None else C.byref(scores), C.byref(_heads(out)), _ptr(lse),
                         _ptr(workspace), workspace.numel(), _ptr(err), made=made, home=stream)


class SharedAttentionPlan(_Plan):
    """engram_shared_attention for fixed tensors: one new token q [B, Hq, D] (bf16) of each of B sequences, those of group g
    the rows [groups[g], groups[g + 1]) (int32 [n + 1]), over the group's prefix (prefix_table int32 [n, width], prefix_lens
    int32 [n]) and then over the sequence's own tokens (block_table, seq_lens). The rest as PagedAttentionPlan."""

    def __init__(self, cache: KVCache, q, prefix_table, prefix_lens, groups, block_table, seq_lens, scale=None, cap: float = 0.0,
                 slopes=None, out=None, lse=None, workspace=None, err=None, stream=None):
        B, Hq, _ = _query(cache, q, (torch.bfloat16,))
        _tensor(groups, 1, "groups")
        n = groups.shape[0] - 1
        if n < 0:
            raise ValueError("groups must have an entry for each group, and the end")
        _vector(groups, n + 1, torch.int32, "groups")
        prefix = _paged_seqs(prefix_table, prefix_lens, n, "prefix_table", "prefix_lens")
        seqs = _paged_seqs(block_table, seq_lens, B)
        scores = _scores(cap, slopes, Hq)
        out, lse, workspace, made = _attention_outputs(cache, q, out, lse, workspace, err, stream,
                                                       lambda: shared_workspace(cache, Hq, B, n), prefix_table=prefix_table,
                                                       prefix_lens=prefix_lens, groups=groups, block_table=block_table,
                                                       seq_lens=seq_lens, slopes=slopes)
        self.out, self.lse, self.workspace = out, lse, workspace
        super().__init__("engram_shared_attention", q.device,
                         (cache, q, prefix_table, prefix_lens, groups, block_table, seq_lens, slopes, out, lse, workspace, err),
                         C.byref(cache._c), C.byref(prefix), _ptr(groups), C.byref(seqs), C.byref(_heads(q)), _scale(cache, scale),
                         None if scores is None else C.byref(scores), C.byref(_heads(out)), _ptr(lse), _ptr(workspace),
                         workspace.numel(), _ptr(err), made=made, home=stream)


# ---------------------------------------------------------------------------------------------
# calls
# ---------------------------------------------------------------------------------------------

def engram_qk_norm_rope(nr: NormRope, q, k, positions, q_out=None, k_out=None, err=None, stream=None):
    """Norm and rotation of query and key rows; returns (q_out, k_out). See QKNormRopePlan."""
    plan = QKNormRopePlan(nr, q, k, positions, q_out, k_out, err, stream)
    plan.run(stream)
    return plan.q_out, plan.k_out


def engram_kv_write(cache: KVCache, k, v, slots, err=None, stream=None):
    """Key and value rows to their slots of the cache. See KVWritePlan."""
    KVWritePlan(cache, k, v, slots, err).run(stream)


def engram_kv_read(cache: KVCache, slots, k_out=None, v_out=None, err=None, stream=None):
    """The rows at slots; returns (k_out, v_out). See KVReadPlan."""
    plan = KVReadPlan(cache, slots, k_out, v_out, err, stream)
    plan.run(stream)
    return plan.k_out, plan.v_out


def engram_paged_attention(cache: KVCache, q, block_table, seq_lens, scale=None, window: int = 0, out=None, lse=None, workspace=None,
                           err=None, stream=None, cap: float = 0.0, slopes=None):
    """Attention of one token per sequence; returns out, or (out, lse) if lse was asked for. See
    PagedAttentionPlan."""
    plan = PagedAttentionPlan(cache, q, block_table, seq_lens, scale, window, out, lse, workspace, err, stream, cap, slopes)
    plan.run(stream)
    return plan.out if plan.lse is None else (plan.out, plan.lse)


def engram_attention_step(nr: NormRope, cache: KVCache, q, k, v, positions, slots, block_table, seq_lens, scale=None, window: int = 0,
                          out=None, lse=None, workspace=None, err=None, stream=None, cap: float = 0.0, slopes=None):
    """One decode step of a layer's attention; returns out, or (out, lse). See AttentionStepPlan."""
    plan = AttentionStepPlan(nr, cache, q, k, v, positions, slots, block_table, seq_lens, scale, window, out, lse, workspace, err,
                             stream, cap, slopes)
    plan.run(stream)
    return plan.out if plan.lse is None else (plan.out, plan.lse)


def engram_prompt_attention(cache: KVCache, q, cu_seqlens, block_table, seq_lens, scale=None, causal: bool = True, window: int = 0,
                            doc_starts=None, prefix_ends=None, cap: float = 0.0, slopes=None, out=None, lse=None, workspace=None,
                            err=None, stream=None):
    """Attention of all new tokens of ragged sequences; returns out, or (out, lse). See PromptAttentionPlan."""
    plan = PromptAttentionPlan(cache, q, cu_seqlens, block_table, seq_lens, scale, causal, window, doc_starts, prefix_ends, cap, slopes,
                               out, lse, workspace, err, stream)
    plan.run(stream)
    return plan.out if plan.lse is None else (plan.out, plan.lse)


def engram_shared_attention(cache: KVCache, q, prefix_table, prefix_lens, groups, block_table, seq_lens, scale=None, cap: float = 0.0,
                            slopes=None, out=None, lse=None, workspace=None, err=None, stream=None):
    """Attention of one token per sequence where groups share a prefix; returns out, or (out, lse). See SharedAttentionPlan."""
    plan = SharedAttentionPlan(cache, q, prefix_table, prefix_lens, groups, block_table, seq_lens, scale, cap, slopes, out, lse,
                               workspace, err, stream)
    plan.run(stream)
    return plan.out if plan.lse is None else (plan.out, plan.lse)
