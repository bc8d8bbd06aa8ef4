"""Shared helpers of the attention operators' GPU tests: paged caches in every layout, filled so that
nothing outside a sequence's tokens may be used."""
import numpy as np
import torch

DEV = "cuda"
P_REL = {"bf16": 2.0 ** -16, "fp8": 2.0 ** -11}              # rounding of the weights (two bf16; one f16)
Q_REL = {("bf16", torch.bfloat16): 0.0, ("fp8", torch.bfloat16): 0.0,
         ("bf16", torch.float32): 2.0 ** -16, ("fp8", torch.float32): 2.0 ** -21}   # two bf16; two f16
U_BF16 = 2.0 ** -8                                            # half a step of bf16, relative


def pkg():
    import engram_gram_hash_02_gb300 as E
    return E


def empty_cache(pages, page, Hk, D, fmt, layout="hnd"):
    """A cache whose memory is all NaN (bf16), or NaN codes with scale bytes 255 (FP8)."""
    E = pkg()
    shape = (pages, Hk, page, D) if layout != "nhd" else (pages, page, Hk, D)
    dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
    junk = float("nan") if fmt == "bf16" else 0x7F
    if layout == "padded":                                   # k and v of a page side by side, rows longer than D
        both = torch.full((pages, 2, Hk, page, D + 32), junk, dtype=dtype, device=DEV)
        k, v = both[:, 0, :, :, :D], both[:, 1, :, :, :D]
    else:
        k, v = (torch.full(shape, junk, dtype=dtype, device=DEV) for _ in range(2))
        if layout == "nhd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
    if fmt == "bf16":
        return E.KVCache(k, v)
    words = (*shape[:3], 4 * -(-D // 128))
    ks, vs = (torch.full(words, 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    return E.KVCache(k, v, *((ks.transpose(1, 2), vs.transpose(1, 2)) if layout == "nhd" else (ks, vs)))


def tables(lens, page, rng, spare=2, width=None):
    """Pages of every sequence at random places; entries a sequence does not use are out of range."""
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), width or max(max(need), 1)), 2 ** 30, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def slots_of(table, b, first, last, page):
    pos = np.arange(first, last)
    return table[b, pos // page].astype(np.int64) * page + pos % page


def dense(cache, slots):
    """fp64 rows [n, Hk, D] of k and v at slots, decoded by the oracle."""
    from oracle import attention_oracle as A
    page = cache.page_size
    p, at = torch.from_numpy(slots // page).to(DEV), torch.from_numpy(slots % page).to(DEV)
    got = []
    for x, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        rows = x[p, :, at]
        if cache.fmt == "bf16":
            got.append(rows.double().cpu().numpy())
        else:
            got.append(A.fp8_decode(rows.cpu().numpy(), s[p, :, at][..., :cache.head_dim // 32].cpu().numpy()))
    return got


def filled(lens, page, Hk, D, fmt, seed, layout="hnd", spread=0.0):
    """A cache with the rows of len tokens per sequence (values ~N(0,1), times 2^N(0, spread)), its page
    table (numpy) and everything else in it unusable."""
    E = pkg()
    rng = np.random.default_rng(seed)
    table, pages = tables(lens, page, rng)
    cache = empty_cache(pages, page, Hk, D, fmt, layout)
    slots = np.concatenate([slots_of(table, b, 0, n, page) for b, n in enumerate(lens)] + [np.zeros(0, np.int64)])
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = [torch.randn((len(slots), Hk, D), generator=g, device=DEV) for _ in range(2)]
    if spread:
        rows[1] *= torch.exp2(spread * torch.randn((len(slots), Hk, 1), generator=g, device=DEV))
    if len(slots):
        E.engram_kv_write(cache, *rows, torch.from_numpy(slots).to(DEV))
    return cache, table


def check_attention(cache, table, lens, q, out, lse, scale, window=0, hidden=None):
    """out and lse against the oracle, every element within the bound; `hidden`: keys to leave out per b."""
    from oracle import attention_oracle as A
    q64, got, got_lse = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        pos = np.arange(first, n)
        if hidden is not None:
            pos = pos[~np.isin(pos, hidden[b])]
        slots = table[b, pos // cache.page_size].astype(np.int64) * cache.page_size + pos % cache.page_size
        k, v = dense(cache, slots)
        ref, ref_lse, tol, tol_lse = A.attention(q64[b], k, v, scale, Q_REL[cache.fmt, q.dtype], P_REL[cache.fmt])
        if len(pos) == 0:
            assert not got[b].any() and np.all(got_lse[b] == -np.inf), f"sequence {b} is empty"
            continue
        err = np.abs(got[b] - ref)
        assert np.isfinite(got[b]).all(), f"sequence {b}"
        worst = (err - (U_BF16 * np.abs(ref) + tol)).max()
        assert worst <= 0, f"sequence {b} of {n}: out past its bound by {worst:.3g} (largest error {err.max():.3g})"
        lerr = np.abs(got_lse[b] - ref_lse)
        assert (lerr <= tol_lse).all(), f"sequence {b} of {n}: lse off by {lerr.max():.3g}, bound {tol_lse.min():.3g}"
