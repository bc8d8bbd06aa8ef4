"""The decode step in the forms its own tests leave out: with a window, with heads turned in part (either pairing), over
each cache format; against its parts bit for bit, and against the 64-bit formulas."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests import _attention as H

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hk,G,D,page,window,R,start,inter,dtype", [
    ([1, 7, 20, 21, 300], 2, 4, 128, 16, 20, 128, 0, False, torch.bfloat16),
    ([1, 64, 129, 1000], 1, 16, 64, 24, 128, 32, 32, False, torch.float32),
    ([5, 33, 700], 2, 5, 256, 8, 1, 64, 192, True, torch.bfloat16),
    ([2, 2049, 90], 3, 8, 96, 64, 0, 32, 0, True, torch.float32),
    ([3, 500] * 20, 2, 12, 192, 16, 100, 16, 8, False, torch.bfloat16),
    ([40, 1, 128], 1, 1, 32, 1, 0, 8, 16, True, torch.float32),
])
def test_step_with_a_window_and_heads_turned_in_part(fmt, lens, Hk, G, D, page, window, R, start, inter, dtype):
    E = H.pkg()
    B, Hq = len(lens), Hk * G
    rng = np.random.default_rng(D + R)
    g = torch.Generator(device=DEV).manual_seed(D + R)
    table, pages = H.tables(lens, page, rng)
    cache = H.empty_cache(pages, page, Hk, D, fmt)
    old = np.concatenate([H.slots_of(table, b, 0, n - 1, page) for b, n in enumerate(lens)])
    E.engram_kv_write(cache, *(torch.randn((len(old), Hk, D), generator=g, device=DEV) for _ in range(2)), torch.from_numpy(old).to(DEV))
    q, k, v = ((3 * torch.randn((B, h, D), generator=g, device=DEV)).to(dtype) for h in (Hq, Hk, Hk))
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2))
    angles = A.rope_angles(max(lens), R)
    nr = E.NormRope(qw, kw, 1e-6, torch.from_numpy(angles).to(DEV), start=start, interleaved=inter)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pos, bt = sl - 1, torch.from_numpy(table).to(DEV)
    slots = torch.tensor([int(H.slots_of(table, b, n - 1, n, page)[0]) for b, n in enumerate(lens)], device=DEV)

    parts = E.KVCache(*(None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)))
    q32, k32 = (torch.empty(x.shape, dtype=torch.float32, device=DEV) for x in (q, k))
    E.engram_qk_norm_rope(nr, q, k, pos, q32, k32)
    for x, w, got in ((q, qw, q32), (k, kw, k32)):
        ref = A.norm_rope(x.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6, angles, pos.cpu().numpy(), start, inter)
        # mean of D squares, rsqrt and four products (40 * 2^-24 at most), then the turn's two products
        assert (np.abs(got.double().cpu().numpy() - ref) <= 64 * 2.0 ** -24 * 2 ** 0.5 * np.abs(ref).max(-1, keepdims=True)).all()
    E.engram_kv_write(parts, k32, v.float(), slots)
    want, want_lse = E.engram_paged_attention(parts, q32, bt, sl, window=window, lse=True)

    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = E.engram_attention_step(nr, cache, q, k, v, pos, slots, bt, sl, window=window, lse=True, err=err)
    assert int(err) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    for a, b in ((cache.k, parts.k), (cache.v, parts.v), (cache.k_scales, parts.k_scales), (cache.v_scales, parts.v_scales)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    H.check_attention(cache, table, lens, q32, out, lse, D ** -0.5, window)
