"""Attention over an FP8 cache whose value rows are of uneven size: blocks of one row far apart, blocks and rows of
zeros, caches with one scale for everything. Every output element is held to the bound that the weights' f16 gives it,
in terms of its own block (derived in `bound`)."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests import _attention as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [(64, 4, "bf16"), (64, 16, "f32"), (128, 4, "f32"), (128, 12, "bf16"), (160, 8, "bf16"), (256, 4, "bf16"), (256, 16, "f32")]
LENS = [1, 40, 130, 3000]
PAGE, HK = 16, 2


def bound(q, k, codes, exps, scale, q_dtype):
    """The oracle's (out, lse) of one sequence and the errors they may have: q [Hq, D], k [n, Hk, D], value codes as
    numbers and their scales' exponents [n, Hk, D].

    Key j enters a block as f16(f16(w_j) * 2^(exponent - e_j)), w_j = 2^15 at the largest p_j 2^e_j there is, e_j the
    largest exponent of row j's blocks that are not zero (-64 at least). Both roundings are 2^-11 relative (P_REL) or,
    below 2^-14, 2^-25 absolute: together 2^-24 of w's unit, 2^-39 max_i(p_i 2^e_i), for every code."""
    v = codes * np.exp2(exps)
    out, lse, tol, tol_lse = A.attention(q, k, v, scale, H.Q_REL["fp8", q_dtype], H.P_REL["fp8"])
    n, Hk, D = k.shape
    e = np.where(codes.reshape(n, Hk, -1, 32).any(-1), exps.reshape(n, Hk, -1, 32)[..., 0], -np.inf).max(-1)
    e = np.maximum(e, -64.0)
    for h in range(len(q)):
        hk = h * Hk // len(q)
        s = k[:, hk] @ q[h] * scale
        top = np.exp(s - lse[h] + np.log(2.0) * e[:, hk]).max()
        tol[h] += 2.0 ** -39 * top * np.abs(codes[:, hk]).sum(0)
    return out, lse, tol, tol_lse


def cached(cache, table, b, n):
    """Keys, value codes as numbers and exponents [n, Hk, D] of a sequence, in 64 bits."""
    slots = H.slots_of(table, b, 0, n, PAGE)
    k, _ = H.dense(cache, slots)
    p, at = torch.from_numpy(slots // PAGE).to(DEV), torch.from_numpy(slots % PAGE).to(DEV)
    bytes_ = cache.v_scales[p, :, at][..., :cache.head_dim // 32].cpu().numpy()
    codes = A.fp8_decode(cache.v[p, :, at].cpu().numpy(), np.full_like(bytes_, 127))
    return k, codes, np.repeat(bytes_.astype(np.float64) - 127, 32, -1)


def attend(lens, D, G, q_type, make, unit=False, scale=None):
    """`make(g, n)` gives the value rows [n, HK, D] of one sequence and what is added to its scores [n] (nats). The
    queries share a direction, along which a key's share is what is to be added."""
    E = H.pkg()
    rng = np.random.default_rng(D + G)
    g = torch.Generator(device=DEV).manual_seed(D + G)
    table, pages = H.tables(lens, PAGE, rng)
    cache = H.empty_cache(pages, PAGE, HK, D, "fp8")
    scale = D ** -0.5 if scale is None else scale
    way = torch.where(torch.rand(D, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    dtype = torch.float32 if q_type == "f32" else torch.bfloat16
    q = (way + 0.25 * torch.randn((len(lens), HK * G, D), generator=g, device=DEV)).to(dtype)
    for b, n in enumerate(lens):
        v, extra = make(g, n)
        noise = 0.25 * torch.randn((n, HK, D), generator=g, device=DEV)
        k = noise + (extra / (scale * D))[:, None, None] * way
        slots = torch.from_numpy(H.slots_of(table, b, 0, n, PAGE)).to(DEV)
        E.engram_kv_write(cache, k, v, slots)
        if unit:                                             # plain e4m3 values, every scale 1
            p, at = slots // PAGE, slots % PAGE
            cache.v[p, :, at] = v.to(torch.float8_e4m3fn).view(torch.uint8)
            cache.v_scales[p, :, at] = 127
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = E.engram_paged_attention(cache, q, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                        scale=scale, lse=True, err=err)
    assert int(err) == 0
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        ref, ref_lse, tol, tol_lse = bound(q[b].double().cpu().numpy(), *cached(cache, table, b, n), scale, dtype)
        e = np.abs(got[b] - ref)
        past = e - (H.U_BF16 * np.abs(ref) + tol)
        assert np.isfinite(got[b]).all() and past.max() <= 0, \
            f"sequence {b} of {n}: {(past > 0).mean():.2%} of the values past their bound, one by {(e / (np.abs(ref) + 1e-300))[past > 0].max():.2g} of itself"
        assert (np.abs(got_lse[b] - ref_lse) <= tol_lse).all(), f"sequence {b}: lse"


def randn(g, n, D):
    return torch.randn((n, HK, D), generator=g, device=DEV)


def nothing(n):
    return torch.zeros(n, device=DEV)


@pytest.mark.parametrize("apart", [5, 12, 20])
@pytest.mark.parametrize("D,G,q_type", FORMS)
def test_blocks_of_a_row_far_apart(D, G, q_type, apart):
    def make(g, n):
        down = torch.rand((n, HK, D // 32, 1), generator=g, device=DEV) * apart
        down[:, :, 0] = apart                                # one block is small in every row
        down[:, :, 1] = 0
        return (randn(g, n, D).unflatten(-1, (-1, 32)) * torch.exp2(-down)).flatten(-2), nothing(n)
    attend(LENS, D, G, q_type, make)


@pytest.mark.parametrize("size", [1.0, 1e-5, 1e-8])
@pytest.mark.parametrize("D,G,q_type", FORMS)
def test_a_block_of_zeros_costs_the_other_blocks_nothing(D, G, q_type, size):
    def make(g, n):
        v = size * randn(g, n, D)
        zero = torch.randint(0, D // 32, (n, HK, 1), generator=g, device=DEV) == torch.arange(D // 32, device=DEV)
        return v.unflatten(-1, (-1, 32)).masked_fill(zero.unsqueeze(-1), 0.0).flatten(-2), nothing(n)
    attend(LENS, D, G, q_type, make)


@pytest.mark.parametrize("above,size", [(10.0, 1.0), (14.0, 1e-2), (18.0, 1e-2), (18.0, 1e-5), (40.0, 1.0)])
@pytest.mark.parametrize("D,G,q_type", FORMS)
def test_a_zero_row_that_takes_the_weight(D, G, q_type, above, size):
    def make(g, n):
        v, extra = size * randn(g, n, D), nothing(n)
        v[n // 2] = -0.0 if n % 3 else 0.0
        extra[n // 2] = above
        return v, extra
    attend(LENS, D, G, q_type, make)


@pytest.mark.parametrize("D,G,q_type", FORMS)
def test_values_that_are_all_zero(D, G, q_type):
    attend([1, 33, 700], D, G, q_type, lambda g, n: (torch.zeros((n, HK, D), device=DEV), nothing(n)))


@pytest.mark.parametrize("D,G,q_type", FORMS)
def test_one_scale_for_every_value(D, G, q_type):
    def make(g, n):
        v, extra = randn(g, n, D), nothing(n)
        v[n // 2] = 0
        v[:, :, 32:64] *= 2.0 ** -5
        v[1::3, :, :32] = 0
        extra[n // 2] = 16.0
        return v, extra
    attend(LENS, D, G, q_type, make, unit=True)


def test_a_block_of_one_value_is_not_taken_for_zeros():
    """Scale 1, as a block of zeros has it, and one value, in each place of the 32."""
    D, G = 128, 4

    def make(g, n):
        v = torch.zeros((n, HK, D), device=DEV)
        i = torch.arange(n, device=DEV)
        v[i, :, i % D] = 300.0                               # amax in (224, 448]: its block's scale is 1, as a zero block's
        v[i, :, (i * 7 + 64) % D] += 1e-3
        return v, nothing(n)
    attend([1, 130, 600], D, G, "bf16", make)
