"""The attention operators through the C ABI against the 64-bit oracle: norms with rotation, the paged
cache's rows, attention of one token per sequence, and the decode step that joins them. Caches are filled
with NaN wherever no token lies. Bounds come from the formulas' rounding (see the oracle), not from runs."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests import _attention as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
ZERO = 16384            # ENGRAM_ATTENTION_ZERO_BYTES


def E():
    return H.pkg()


def randn(g, shape, dtype=torch.float32, std=1.0):
    return (std * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------ norms and rotation

NORM_CASES = [
    # T, Hq, Hk, D, R, start, interleaved, in, out, layout
    (1, 32, 8, 128, 128, 0, False, "bf16", "bf16", "plain"),
    (1, 1, 1, 8, 0, 0, False, "f32", "f32", "plain"),
    (7, 3, 1, 64, 64, 0, True, "bf16", "f32", "plain"),
    (33, 5, 2, 96, 32, 64, False, "f32", "bf16", "packed"),
    (130, 4, 4, 256, 64, 192, True, "f32", "f32", "packed"),
    (129, 2, 1, 72, 16, 8, False, "bf16", "bf16", "heads_first"),
    (5, 9, 3, 40, 8, 32, True, "f32", "bf16", "in_place_rows"),
    (4097, 20, 4, 128, 128, 0, False, "bf16", "bf16", "plain"),
    (2500, 16, 16, 256, 256, 0, True, "f32", "bf16", "plain"),
    (3000, 12, 3, 64, 32, 0, False, "bf16", "bf16", "packed"),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,start,inter,tin,tout,layout", NORM_CASES)
def test_qk_norm_rope_matches_the_formula(T, Hq, Hk, D, R, start, inter, tin, tout, layout):
    g = torch.Generator(device=DEV).manual_seed(T + D)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    if layout == "packed":                                   # [q | k | v] in one row
        rows = randn(g, (T, Hq + 2 * Hk, D), dt[tin], 3.0)
        q, k = rows[:, :Hq], rows[:, Hq:Hq + Hk]
    elif layout == "heads_first":                            # [heads, T, D]
        q, k = (randn(g, (h, T, D), dt[tin], 0.02).transpose(0, 1) for h in (Hq, Hk))
    else:
        q, k = (randn(g, (T, h, D), dt[tin], 1.0) for h in (Hq, Hk))
    q[-1, -1] = 0                                            # a row of zeros stays zeros
    qw, kw = ((1 + randn(g, (D,), std=0.1)).bfloat16() for _ in range(2))
    eps, rows_n = 1e-6, 5000
    table = A.rope_angles(rows_n, R) if R else None
    pos = torch.randint(0, rows_n, (T,), generator=g, device=DEV, dtype=torch.int32)
    nr = E().NormRope(qw, kw, eps, None if table is None else torch.from_numpy(table).to(DEV), start=start, interleaved=inter)
    refs = [A.norm_rope(x.double().cpu().numpy(), w.double().cpu().numpy(), eps, table, pos.cpu().numpy(), start, inter)
            for x, w in ((q, qw), (k, kw))]
    err = word()
    outs = [torch.full((T, h, D), float("nan"), dtype=dt[tout], device=DEV) for h in (Hq, Hk)]
    if layout == "heads_first":
        outs = [torch.full((h, T, D), float("nan"), dtype=dt[tout], device=DEV).transpose(0, 1) for h in (Hq, Hk)]
    got = E().engram_qk_norm_rope(nr, q, k, pos, *outs, err=err)
    assert got[0] is outs[0] and got[1] is outs[1] and int(err) == 0
    for x, ref in zip(outs, refs):
        # mean of D squares, rsqrt and four products (40 * 2^-24 at most), then the turn's two products
        tol = 64 * 2.0 ** -24 * np.abs(ref).max(-1, keepdims=True) * 2 ** 0.5 + (H.U_BF16 * np.abs(ref) if tout == "bf16" else 0)
        e = np.abs(x.double().cpu().numpy() - ref)
        assert (e <= tol).all(), f"largest error {e.max():.3g}"


def test_qk_norm_rope_in_place_one_sided_and_without_parts():
    g = torch.Generator(device=DEV).manual_seed(3)
    T, D = 45, 128
    q, k = randn(g, (T, 8, D), torch.bfloat16), randn(g, (T, 2, D), torch.bfloat16)
    w = (1 + randn(g, (D,), std=0.1)).bfloat16()
    table = torch.from_numpy(A.rope_angles(T, 64)).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    nr = E().NormRope(w, w, 1e-5, table, start=64)
    want = E().engram_qk_norm_rope(nr, q, k, pos)
    only_q = E().engram_qk_norm_rope(nr, q, None, pos)
    only_k = E().engram_qk_norm_rope(nr, None, k, pos)
    assert torch.equal(only_q[0], want[0]) and only_q[1] is None and torch.equal(only_k[1], want[1])
    q2, k2 = q.clone(), k.clone()
    E().engram_qk_norm_rope(nr, q2, k2, pos, q2, k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    # neither norm nor rotation: a copy; no rotation: no positions needed
    same = E().engram_qk_norm_rope(E().NormRope(None, None, 0.0, None), q, k, None)
    assert torch.equal(same[0], q) and torch.equal(same[1], k)
    # no tokens
    none = E().engram_qk_norm_rope(nr, q[:0], k[:0], pos[:0])
    assert none[0].shape == (0, 8, D)


def test_positions_outside_the_table_take_the_nearest_row_and_are_reported():
    g = torch.Generator(device=DEV).manual_seed(4)
    q = randn(g, (3, 2, 64), torch.float32)
    nr = E().NormRope(None, None, 0.0, torch.from_numpy(A.rope_angles(10, 64)).to(DEV))
    err = word()
    out = [torch.empty_like(q) for _ in range(2)]
    E().engram_qk_norm_rope(nr, q, None, torch.tensor([-5, 10, 3], dtype=torch.int32, device=DEV), out[0], err=err)
    E().engram_qk_norm_rope(nr, q, None, torch.tensor([0, 9, 3], dtype=torch.int32, device=DEV), out[1])
    assert torch.equal(out[0], out[1]) and int(err) == E().ERR_POSITION
    assert E().sync_status(err) == -3


# -------------------------------------------------------------------------------------- cache rows

@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,Hk,D,page,layout,dtype", [
    (1, 1, 32, 1, "hnd", torch.bfloat16),
    (77, 8, 128, 16, "hnd", torch.bfloat16),
    (300, 3, 96, 7, "nhd", torch.float32),
    (65, 2, 256, 24, "padded", torch.bfloat16),
    (5000, 5, 64, 64, "nhd", torch.bfloat16),
    (4100, 8, 192, 32, "hnd", torch.float32),
])
def test_written_rows_are_the_formula_bit_for_bit_and_read_back(fmt, T, Hk, D, page, layout, dtype):
    rng = np.random.default_rng(T)
    g = torch.Generator(device=DEV).manual_seed(T)
    pages = -(-T // page) + 2
    cache = H.empty_cache(pages, page, Hk, D, fmt, layout)
    k, v = (randn(g, (T, Hk, D)) * torch.exp2(randn(g, (T, Hk, 1), std=20.0)) for _ in range(2))
    k, v = k.to(dtype), v.to(dtype)
    k[0] = 0
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    skip = rng.random(T) < 0.1
    given = np.where(skip, -1 - rng.integers(0, 5, T), slots)
    before = [x.clone() for x in (cache.k, cache.v)]
    err = word()
    E().engram_kv_write(cache, k, v, torch.from_numpy(given).to(DEV), err=err)
    keep = np.flatnonzero(~skip)
    p, at = torch.from_numpy(slots[keep] // page).to(DEV), torch.from_numpy(slots[keep] % page).to(DEV)
    for x, rows, scales, old in ((k, cache.k, cache.k_scales, before[0]), (v, cache.v, cache.v_scales, before[1])):
        if fmt == "bf16":
            assert torch.equal(rows[p, :, at], x[keep].bfloat16())
        else:
            codes, bytes_ = A.fp8_encode(x[keep].float().cpu().numpy())
            assert np.array_equal(rows[p, :, at].cpu().numpy(), codes)
            assert np.array_equal(scales[p, :, at].cpu().numpy()[..., :D // 32], bytes_)
        # nothing else was touched
        rest = torch.ones((pages, page), dtype=torch.bool, device=DEV)
        rest[p, at] = False
        pr, ar = rest.nonzero(as_tuple=True)
        assert torch.equal(rows[pr, :, ar].contiguous().view(torch.uint8), old[pr, :, ar].contiguous().view(torch.uint8))
    for out in (torch.float32, torch.bfloat16):
        outs = [torch.full((T, Hk, D), 7.0, dtype=out, device=DEV) for _ in range(2)]
        E().engram_kv_read(cache, torch.from_numpy(given).to(DEV), *outs, err=err)
        for x, rows, scales in ((outs[0], cache.k, cache.k_scales), (outs[1], cache.v, cache.v_scales)):
            assert not x[np.flatnonzero(skip)].any()
            if fmt == "bf16":
                want = rows[p, :, at].to(out)
            else:
                want = torch.from_numpy(A.fp8_decode(rows[p, :, at].cpu().numpy(),
                                                     scales[p, :, at].cpu().numpy()[..., :D // 32])).to(DEV).to(out)
            assert torch.equal(x[keep], want)
    assert int(err) == 0


def test_fp8_rows_at_the_edges_of_the_format():
    # block maxima at 448 * 2^e and one ulp to either side, ties, subnormals, the smallest scale, NaN, infinities
    D = 64
    rows = np.zeros((14, 2, D), dtype=np.float32)
    for i, e in enumerate((-130, -100, -8, 0, 7, 110)):
        top = np.float32(448.0) * np.float32(2.0) ** np.float32(e)
        rows[i, 0, 0], rows[i, 0, 32] = top, np.nextafter(top, np.float32(np.inf))
        rows[i, 1, 0], rows[i, 1, 32] = np.nextafter(top, np.float32(0)), -top
        rows[i, :, 1:32] = np.linspace(-1, 1, 31, dtype=np.float32) * top
    rows[6, 0, :32] = 448.0                                   # ties between neighbouring codes
    rows[6, 0, 1:32] = (np.arange(31) + 0.5) * 2.0 ** -9
    rows[7, 0, :] = 2.0 ** -149
    rows[8, 0, 5] = np.nan
    rows[9, 0, 5] = np.inf
    rows[9, 0, 6] = 1.0
    rows[10, 1, 40] = -np.inf
    rows[11, 0, :] = np.float32(3.4e38)
    rows[12, 0, 0] = -0.0
    cache = E().KVCache.allocate(2, 8, 2, D, "fp8")
    slots = torch.arange(14, device=DEV)
    x = torch.from_numpy(rows).to(DEV)
    E().engram_kv_write(cache, x, x, slots)
    codes, bytes_ = A.fp8_encode(rows)
    p, at = slots // 8, slots % 8
    assert np.array_equal(cache.k_scales[p, :, at].cpu().numpy()[..., :2], bytes_)
    assert np.array_equal(cache.v[p, :, at].cpu().numpy(), codes)
    back = torch.empty((14, 2, D), dtype=torch.float32, device=DEV)
    E().engram_kv_read(cache, slots, back, torch.empty_like(back))
    back = back.cpu().numpy()
    with np.errstate(over="ignore"):
        want = A.fp8_decode(codes, bytes_).astype(np.float32)
    assert np.array_equal(back, want, equal_nan=True)
    assert np.isnan(back[8, 0, 5]) and back[9, 0, 5] == np.inf and back[10, 1, 40] == -np.inf and back[9, 0, 6] == 0
    # written once more from the values read back: the same rows
    fine = [i for i in range(14) if np.isfinite(back[i]).all()]
    again, again_bytes = A.fp8_encode(back[fine])
    assert np.array_equal(A.fp8_decode(again, again_bytes), back[fine])


def test_slots_past_the_cache_are_reported():
    cache = E().KVCache.allocate(3, 4, 1, 32)
    k = torch.ones((3, 1, 32), dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([0, 12, 2 ** 40], device=DEV)
    err = word()
    E().engram_kv_write(cache, k, k, slots, err=err)
    assert int(err) == E().ERR_SLOT and float(cache.k.float().sum()) == 32
    err.zero_()
    k_out, v_out = E().engram_kv_read(cache, slots, err=err)
    assert int(err) == E().ERR_SLOT and float(k_out.float().sum()) == 32 and not v_out[1:].any()
    err.zero_()
    E().engram_kv_write(cache, k[:0], k[:0], slots[:0], err=err)
    assert int(err) == 0


# --------------------------------------------------------------------------------------- attention

RAGGED = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500, 0]
ATTENTION_CASES = [
    # lens, Hk, G, D, page, window, q type, layout
    ([1], 1, 1, 32, 1, 0, "bf16", "hnd"),
    (RAGGED, 2, 4, 128, 16, 0, "bf16", "hnd"),
    (RAGGED, 1, 8, 64, 7, 0, "f32", "nhd"),
    (RAGGED, 3, 3, 96, 24, 0, "bf16", "padded"),
    (RAGGED, 2, 5, 256, 200, 0, "bf16", "hnd"),
    (RAGGED, 1, 16, 128, 64, 0, "f32", "hnd"),
    (RAGGED, 2, 9, 192, 32, 0, "bf16", "nhd"),
    (RAGGED, 1, 17, 64, 16, 0, "bf16", "hnd"),
    (RAGGED, 1, 40, 256, 16, 0, "f32", "hnd"),
    (RAGGED, 4, 1, 160, 8, 0, "f32", "nhd"),
    (RAGGED, 2, 2, 64, 24, 20, "bf16", "hnd"),
    (RAGGED, 1, 8, 128, 16, 1, "bf16", "hnd"),
    ([1000, 3, 777, 2049], 2, 12, 128, 48, 300, "f32", "padded"),
    ([5000], 1, 8, 128, 64, 0, "bf16", "hnd"),
    ([20011], 1, 16, 256, 64, 0, "f32", "hnd"),
    ([70001, 1], 2, 4, 64, 128, 0, "bf16", "nhd"),
    (list(range(300)), 1, 2, 64, 16, 0, "bf16", "hnd"),
    ([130] * 200, 4, 1, 128, 16, 0, "bf16", "hnd"),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hk,G,D,page,window,tq,layout", ATTENTION_CASES)
def test_paged_attention_matches_the_formula(lens, Hk, G, D, page, window, tq, layout, fmt):
    seed = sum(lens) + D + G
    cache, table = H.filled(lens, page, Hk, D, fmt, seed, layout, spread=3.0)
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hq = len(lens), Hk * G
    q = randn(g, (B, Hq, D), torch.float32 if tq == "f32" else torch.bfloat16, 2.0)
    out = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, Hq), float("nan"), device=DEV)
    ws = E().attention_workspace(cache, Hq, B)
    ws[ZERO:] = 0xFF                                          # only the first words need to be zero
    err = word()
    scale = D ** -0.5
    plan = E().PagedAttentionPlan(cache, q, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                  window=window, out=out, lse=lse, workspace=ws, err=err)
    plan.run()
    assert int(err) == 0 and not ws[:ZERO].any()
    H.check_attention(cache, table, lens, q, out, lse, scale, window)
    # once more: the same bits
    first = out.clone(), lse.clone()
    out.fill_(float("nan"))
    plan.run()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and not ws[:ZERO].any()


def test_attention_strided_rows_default_outputs_and_scales():
    lens, Hk, G, D, page = [70, 0, 9], 2, 3, 64, 16
    cache, table = H.filled(lens, page, Hk, D, "bf16", 5)
    g = torch.Generator(device=DEV).manual_seed(5)
    packed = randn(g, (3, Hk * G + 2 * Hk, D), torch.bfloat16)
    q = packed[:, :Hk * G]
    wide = torch.zeros((3, 7), dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = torch.from_numpy(table).to(DEV)
    bt = wide[:, :table.shape[1]]                            # rows of a wider table
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, lse = E().engram_paged_attention(cache, q, bt, sl, lse=True)
    H.check_attention(cache, table, lens, q, want, lse, D ** -0.5)
    # heads first, and only the output
    out = torch.empty((Hk * G, 3, D), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert E().engram_paged_attention(cache, q, bt, sl, out=out) is out
    assert torch.equal(out, want)
    for scale in (0.0, -0.3, 1.0):
        got, lse = E().engram_paged_attention(cache, q, bt, sl, scale=scale, lse=True)
        H.check_attention(cache, table, lens, q, got, lse, scale)
    # no sequences
    assert E().engram_paged_attention(cache, q[:0], bt[:0], sl[:0]).shape == (0, Hk * G, D)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_bad_pages_and_lengths_hide_their_tokens_and_are_reported(fmt):
    lens, page = [100, 50, 40], 16
    cache, table = H.filled(lens, page, 2, 64, fmt, 9)
    q = randn(torch.Generator(device=DEV).manual_seed(9), (3, 4, 64), torch.bfloat16)
    bad = table.copy()
    bad[0, 1], bad[0, 4], bad[2, :] = -1, 2 ** 31 - 1, cache.num_pages
    err = word()
    out, lse = E().engram_paged_attention(cache, q, torch.from_numpy(bad).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                          lse=True, err=err)
    assert int(err) == E().ERR_PAGE
    hidden = [list(range(16, 32)) + list(range(64, 80)), [], list(range(40))]
    H.check_attention(cache, table, lens, q, out, lse, 0.125, hidden=hidden)
    # lengths below 0 are empty, lengths past the table end with it
    err.zero_()
    said = torch.tensor([100, -3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    full = [100, 0, 112]
    cache, table = H.filled(full, page, 2, 64, fmt, 10)
    out, lse = E().engram_paged_attention(cache, q, torch.from_numpy(table).to(DEV), said, lse=True, err=err)
    assert int(err) == E().ERR_SEQ_LEN
    H.check_attention(cache, table, full, q, out, lse, 0.125)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8), (256, 16)])
def test_scores_far_apart_infinite_and_undefined(fmt, D, G):
    lens, page = [200, 200, 200, 200], 16
    cache, table = H.filled(lens, page, 1, D, fmt, 11, spread=4.0)   # value rows over 2^±12
    g = torch.Generator(device=DEV).manual_seed(11)
    q = randn(g, (4, G, D), torch.bfloat16, 30.0)                     # nearly one key takes all
    bt, sl = torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = E().engram_paged_attention(cache, q, bt, sl, lse=True)
    H.check_attention(cache, table, lens, q, out, lse, D ** -0.5)
    # small and large queries
    for std in (2.0 ** -100, 2.0 ** -20, 2.0 ** 12):
        qs = (q * std).bfloat16()
        out, lse = E().engram_paged_attention(cache, qs, bt, sl, scale=1e-3 if std > 1 else 1.0, lse=True)
        H.check_attention(cache, table, lens, qs, out, lse, 1e-3 if std > 1 else 1.0)
    # a NaN or infinite query spoils its own head alone
    qs = q.clone()
    qs[1, 0, 3] = float("nan")
    qs[2, G - 1, 5] = float("inf")
    out2, lse2 = E().engram_paged_attention(cache, qs, bt, sl, lse=True)
    want, _ = E().engram_paged_attention(cache, q, bt, sl, lse=True)
    assert torch.isnan(out2[1, 0]).all() and torch.isnan(lse2[1, 0])
    keep = torch.ones((4, G), dtype=torch.bool, device=DEV)
    keep[1, 0] = keep[2, G - 1] = False
    assert torch.equal(out2[keep], want[keep])


def test_keys_that_are_all_minus_infinity_leave_an_empty_row():
    cache = E().KVCache.allocate(2, 16, 1, 32)
    cache.k.fill_(float("-inf"))
    cache.v.fill_(1.0)
    q = torch.ones((1, 2, 32), dtype=torch.bfloat16, device=DEV)
    bt, sl = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), torch.tensor([20], dtype=torch.int32, device=DEV)
    out, lse = E().engram_paged_attention(cache, q, bt, sl, lse=True)
    assert not out.any() and torch.equal(lse, torch.full_like(lse, float("-inf")))
    cache.k[0, 0, 3] = 0.0                                            # one key with a finite score
    out, lse = E().engram_paged_attention(cache, q, bt, sl, lse=True)
    assert torch.equal(out, torch.ones_like(out)) and float(lse[0, 0]) == 0.0


def test_offsets_past_32_bits():
    # 2^31 values and more than 2^32 bytes on either side; only the last pages hold tokens
    Hk, D, page, lens = 2, 128, 64, [200, 64]
    for fmt in ("bf16", "fp8"):
        pages = (1 << 32) // (Hk * D * page * (2 if fmt == "bf16" else 1)) * 2 + 64
        shape = (pages, Hk, page, D)
        k, v = (torch.empty(shape, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device=DEV) for _ in range(2))
        scales = [torch.empty((*shape[:3], 4), dtype=torch.uint8, device=DEV) for _ in range(2)] if fmt == "fp8" else [None, None]
        cache = E().KVCache(k, v, *scales)
        table = np.array([[pages - 1, pages - 9, pages - 2, pages - 40], [pages - 5, 0, 0, 0]], dtype=np.int32)
        g = torch.Generator(device=DEV).manual_seed(1)
        slots = np.concatenate([H.slots_of(table, b, 0, n, page) for b, n in enumerate(lens)])
        assert slots.max() * Hk * D * (2 if fmt == "bf16" else 1) > 2 ** 32
        rows = [randn(g, (len(slots), Hk, D), torch.bfloat16) for _ in range(2)]
        sd = torch.from_numpy(slots).to(DEV)
        E().engram_kv_write(cache, *rows, sd)
        back = E().engram_kv_read(cache, sd)
        if fmt == "bf16":
            assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])
        else:
            for x, y in zip(back, rows):
                assert np.array_equal(x.double().cpu().numpy(), A.fp8_decode(*A.fp8_encode(y.float().cpu().numpy())))
        q = randn(g, (2, 8, D), torch.bfloat16)
        out, lse = E().engram_paged_attention(cache, q, torch.from_numpy(table).to(DEV),
                                              torch.tensor(lens, dtype=torch.int32, device=DEV), lse=True)
        H.check_attention(cache, table, lens, q, out, lse, D ** -0.5)
        del cache, k, v, scales
        torch.cuda.empty_cache()


def test_one_workspace_serves_calls_of_any_shape_in_order():
    shapes = [([3000, 10], 1, 16, 256), (RAGGED, 2, 4, 64), ([9000], 4, 2, 128), (list(range(1, 200)), 1, 8, 128)]
    made = []
    size = 0
    for i, (lens, Hk, G, D) in enumerate(shapes):
        cache, table = H.filled(lens, 16, Hk, D, ("bf16", "fp8")[i % 2], 20 + i)
        size = max(size, E().attention_workspace_bytes(cache, Hk * G, len(lens)))
        made.append((cache, table, randn(torch.Generator(device=DEV).manual_seed(i), (len(lens), Hk * G, D), torch.bfloat16)))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for (lens, Hk, G, D), (cache, table, q) in zip(shapes, made):
            out, lse = E().engram_paged_attention(cache, q, torch.from_numpy(table).to(DEV),
                                                  torch.tensor(lens, dtype=torch.int32, device=DEV), lse=True, workspace=ws)
            H.check_attention(cache, table, lens, q, out, lse, D ** -0.5)


# -------------------------------------------------------------------------------------------- step

def _step(fmt, lens, Hk, G, D, page, dtype, seed, R=None, window=0):
    """A cache that holds all but the last token of every sequence, and that token's rows."""
    B = len(lens)
    rng = np.random.default_rng(seed)
    table, pages = H.tables(lens, page, rng)
    cache = H.empty_cache(pages, page, Hk, D, fmt)
    g = torch.Generator(device=DEV).manual_seed(seed)
    old = np.concatenate([H.slots_of(table, b, 0, n - 1, page) for b, n in enumerate(lens)])
    if len(old):
        E().engram_kv_write(cache, *(randn(g, (len(old), Hk, D)) for _ in range(2)), torch.from_numpy(old).to(DEV))
    rows = randn(g, (B, (G + 2) * Hk, D), dtype, 3.0)
    q, k, v = rows[:, :G * Hk], rows[:, G * Hk:(G + 1) * Hk], rows[:, (G + 1) * Hk:]
    w = [(1 + randn(g, (D,), std=0.1)).bfloat16() for _ in range(2)]
    nr = E().NormRope(*w, 1e-6, torch.from_numpy(A.rope_angles(max(lens), R or D)).to(DEV))
    slots = torch.tensor([int(H.slots_of(table, b, n - 1, n, page)[0]) for b, n in enumerate(lens)], device=DEV)
    return cache, table, nr, q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV) - 1, slots


def _clone(cache):
    return E().KVCache(*(None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hk,G,D,page,dtype", [
    ([1], 1, 1, 64, 16, torch.bfloat16),
    ([1, 16, 17, 300, 64], 2, 4, 128, 16, torch.bfloat16),
    ([4000, 5], 2, 8, 128, 64, torch.float32),
    ([33] * 70, 1, 12, 256, 8, torch.bfloat16),
])
def test_step_is_its_parts_bit_for_bit_and_matches_the_formula(fmt, lens, Hk, G, D, page, dtype):
    cache, table, nr, q, k, v, pos, slots = _step(fmt, lens, Hk, G, D, page, dtype, 31 + D)
    B = len(lens)
    bt, sl = torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    parts = _clone(cache)
    q32, k32 = (torch.empty(x.shape, dtype=torch.float32, device=DEV) for x in (q, k))
    E().engram_qk_norm_rope(nr, q, k, pos, q32, k32)
    E().engram_kv_write(parts, k32, v.float(), slots)
    want, want_lse = E().engram_paged_attention(parts, q32, bt, sl, lse=True)
    err = word()
    out, lse = E().engram_attention_step(nr, cache, q, k, v, pos, slots, bt, sl, lse=True, err=err)
    assert int(err) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for a, b in ((cache.k, parts.k), (cache.v, parts.v), (cache.k_scales, parts.k_scales), (cache.v_scales, parts.v_scales)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    H.check_attention(cache, table, lens, q32, out, lse, D ** -0.5)


def test_decode_loop_in_a_cuda_graph_on_a_side_stream():
    # ten tokens of three sequences: one captured step, replayed with the state moved on the device
    lens0, Hk, G, D, page, steps = [5, 40, 1], 2, 4, 128, 16, 10
    rng = np.random.default_rng(6)
    table, pages = H.tables([n + steps for n in lens0], page, rng)
    cache = H.empty_cache(pages, page, Hk, D, "fp8")
    g = torch.Generator(device=DEV).manual_seed(6)
    old = np.concatenate([H.slots_of(table, b, 0, n, page) for b, n in enumerate(lens0)])
    E().engram_kv_write(cache, *(randn(g, (len(old), Hk, D)) for _ in range(2)), torch.from_numpy(old).to(DEV))
    nr = E().NormRope(None, None, 0.0, torch.from_numpy(A.rope_angles(64, D)).to(DEV))
    q, k, v = (torch.zeros((3, h, D), dtype=torch.bfloat16, device=DEV) for h in (Hk * G, Hk, Hk))
    pos, sl = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(2))
    slots, bt = torch.full((3,), -1, dtype=torch.int64, device=DEV), torch.from_numpy(table).to(DEV)
    plan = E().AttentionStepPlan(nr, cache, q, k, v, pos, slots, bt, sl, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(side)                                           # once before the capture: attributes are set then
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan.run(side)
    lens = list(lens0)
    for _ in range(steps):
        new = [randn(g, x.shape, torch.bfloat16) for x in (q, k, v)]
        lens = [n + 1 for n in lens]
        for x, y in zip((q, k, v), new):
            x.copy_(y)
        pos.copy_(torch.tensor(lens, dtype=torch.int32) - 1)
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        slots.copy_(torch.tensor([int(H.slots_of(table, b, n - 1, n, page)[0]) for b, n in enumerate(lens)]))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        q32 = torch.empty(q.shape, dtype=torch.float32, device=DEV)
        E().engram_qk_norm_rope(nr, q, None, pos, q32)
        H.check_attention(cache, table, lens, q32, plan.out, plan.lse, D ** -0.5)
        assert not plan.workspace[:ZERO].any()


def test_two_streams_at_once_with_workspaces_of_their_own():
    made = []
    for i in range(2):
        lens = [3000 + 700 * i, 10, 900]
        cache, table = H.filled(lens, 16, 2, 128, "bf16", 40 + i)
        q = randn(torch.Generator(device=DEV).manual_seed(i), (3, 8, 128), torch.bfloat16)
        plan = E().PagedAttentionPlan(cache, q, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                      lse=True)
        made.append((cache, table, lens, q, plan, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for m in made:
            m[4].run(m[5])
    torch.cuda.synchronize()
    for cache, table, lens, q, plan, _ in made:
        H.check_attention(cache, table, lens, q, plan.out, plan.lse, 128 ** -0.5)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_several_new_tokens_of_one_sequence_as_entries_of_the_batch(fmt):
    # entries 0 .. 2 are one sequence's next three tokens, each attending the ones before; entry 3 is another
    Hk, G, D, page = 2, 4, 128, 16
    rng = np.random.default_rng(8)
    owners, pages = H.tables([33, 70], page, rng)
    cache = H.empty_cache(pages, page, Hk, D, fmt)
    g = torch.Generator(device=DEV).manual_seed(8)
    old = np.concatenate([H.slots_of(owners, 0, 0, 30, page), H.slots_of(owners, 1, 0, 69, page)])
    E().engram_kv_write(cache, *(randn(g, (len(old), Hk, D)) for _ in range(2)), torch.from_numpy(old).to(DEV))
    table = owners[[0, 0, 0, 1]]
    lens = [31, 32, 33, 70]
    q, k, v = (randn(g, (4, h, D), torch.bfloat16) for h in (Hk * G, Hk, Hk))
    slots = torch.tensor([int(H.slots_of(table, b, n - 1, n, page)[0]) for b, n in enumerate(lens)], device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nr = E().NormRope(None, None, 0.0, torch.from_numpy(A.rope_angles(80, D)).to(DEV))
    out, lse = E().engram_attention_step(nr, cache, q, k, v, sl - 1, slots, torch.from_numpy(table).to(DEV), sl, lse=True)
    q32 = torch.empty(q.shape, dtype=torch.float32, device=DEV)
    E().engram_qk_norm_rope(nr, q, None, sl - 1, q32)
    H.check_attention(cache, table, lens, q32, out, lse, D ** -0.5)


def test_a_table_without_columns_leaves_every_sequence_empty():
    cache = E().KVCache.allocate(1, 16, 1, 64)
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    err = word()
    out, lse = E().engram_paged_attention(cache, q, torch.zeros((3, 0), dtype=torch.int32, device=DEV),
                                          torch.tensor([0, 5, 0], dtype=torch.int32, device=DEV), lse=True, err=err)
    assert not out.any() and bool(torch.isinf(lse).all()) and int(err) == E().ERR_SEQ_LEN


def test_calls_from_plain_c(tmp_path):
    """tests/c/attention_c_abi.c, built with the host C compiler against include/engram.h."""
    import os
    import shutil
    import subprocess
    from engram_gram_hash_02_gb300 import binding, build
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    binding.lib()
    libdir = os.path.dirname(os.path.abspath(binding.LIB_PATH))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "attention_c_abi.c")
    exe = str(tmp_path / "attention_c_abi")
    subprocess.run([cc, "-std=c99", "-O2", "-Wall", "-Werror", "-I", build.INCLUDE, "-I", os.path.join(cuda, "include"), src, "-L", libdir,
                    "-lengram", "-L", os.path.join(cuda, "lib64"), "-lcudart", "-lm", f"-Wl,-rpath,{libdir}",
                    f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}", "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
