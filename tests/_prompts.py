"""Shared helpers of the GPU tests of prompts, forms of scores and shared prefixes."""
import numpy as np
import torch

from tests import _attention as H

DEV = "cuda"
# weights are rounded to bf16 in a prompt's and a prefix's products
P_PROMPT = 2.0 ** -8


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device=DEV)


def alibi(Hq):
    return np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq).astype(np.float32)


def rows_of(cache, table, b, n):
    """fp64 keys and values [n, Hk, D] of a sequence's n tokens."""
    return H.dense(cache, H.slots_of(table, b, 0, n, cache.page_size))


def check_rows(got, got_lse, ref, what, widen=0.0):
    """Every element of out and lse within its bound; rows that see nothing are zeros and -inf."""
    out, lse, tol, tol_lse = ref
    empty = np.isneginf(lse)
    assert not got[empty].any() and np.isneginf(got_lse[empty]).all(), f"{what}: rows that see nothing"
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - out)
    worst = (err - (H.U_BF16 * (np.abs(out) + tol) + tol * (1 + widen))).max(initial=0.0)
    assert worst <= 0, f"{what}: out past its bound by {worst:.3g} (largest error {err.max():.3g})"
    with np.errstate(invalid="ignore"):
        lerr = np.where(empty, 0.0, np.abs(got_lse - lse))
    assert (lerr <= tol_lse).all(), f"{what}: lse off by {lerr.max():.3g} (bound {tol_lse[lerr > tol_lse].min():.3g})"


def check_prompt(cache, table, new, lens, q, out, lse, scale, causal=True, window=0, doc_starts=None, prefix_ends=None, cap=0.0,
                 slopes=None, hidden=None, rows=None):
    """Every sequence's rows against the oracle. hidden: keys to leave out per sequence; rows: of these rows only."""
    from oracle import attention_oracle as A
    t0 = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        t = slice(t0, t0 + n)
        at = {k: None if x is None else np.asarray(x)[t] for k, x in (("doc_starts", doc_starts), ("prefix_ends", prefix_ends))}
        p, lo, hi = A.visible(n, length, causal, window, **at)
        j = np.arange(length)
        seen = (j >= lo[:, None]) & (j < hi[:, None])
        if hidden is not None:
            seen &= ~np.isin(j, hidden[b])
        ok = [x for x in range(length) if hidden is None or x not in hidden[b]]
        k, v = (np.zeros((length, cache.kv_heads, cache.head_dim)) for _ in range(2))
        if ok:
            slots = H.slots_of(table, b, 0, length, cache.page_size)[ok]
            k[ok], v[ok] = H.dense(cache, slots)
        k, v = np.nan_to_num(k, posinf=0.0, neginf=0.0), np.nan_to_num(v, posinf=0.0, neginf=0.0)
        ref = A.attention_rows(q[t].double().cpu().numpy(), k, v, seen, p, scale, cap, slopes, p_rel=P_PROMPT)
        got, got_lse = out[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
        if rows is not None:
            keep = np.isin(np.arange(t0, t0 + n), rows)
            ref, got, got_lse = tuple(x[keep] for x in ref), got[keep], got_lse[keep]
        check_rows(got, got_lse, ref, f"sequence {b} of {n} new in {length}")
        t0 += n
