"""The attention operators of a decode layer, in their plain form and through the package's entry points.

Four operators: `norm_rope` (per-head RMS norm of queries and keys with the position rotation), `cache` (rows written to a
paged key-value cache, bf16 or 8-bit, and read back), `attention` (one new token per sequence over the paged cache) and `step`
(norm, rotation, cache write and attention of one token per sequence, as a decode loop calls them).
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one sequence, the latency of a single decode: 32 query heads, 8 key heads of 128
        dict(name="norm_rope_1", op="norm_rope", T=1, Hq=32, Hk=8, D=128, R=128, start=0, interleaved=False, x="bf16", packed=False),
        # eight prompts of 4096 tokens at once
        dict(name="norm_rope_32768", op="norm_rope", T=32768, Hq=32, Hk=8, D=128, R=128, start=0, interleaved=False, x="bf16",
             packed=False),
        # an odd number of prompt tokens straight from an fp32 projection: heads of 256 packed as [q | k | v] in one row, the
        # last 64 values rotated in pairs
        dict(name="norm_rope_fp32_packed", op="norm_rope", T=1777, Hq=20, Hk=4, D=256, R=64, start=192, interleaved=True, x="f32",
             packed=True),
        # the rows of 256 decoding sequences, quantised into their places and read back
        dict(name="cache_fp8_256", op="cache", T=256, Hk=8, D=128, page=64, fmt="fp8", skip=0.0),
        # eight prompts of 4096 tokens, some padded: quantised, and read back for a later chunk of the prompt
        dict(name="cache_fp8_32768", op="cache", T=32768, Hk=8, D=128, page=64, fmt="fp8", skip=0.02),
        # one sequence in its first hundreds of tokens: latency
        dict(name="attention_1x777", op="attention", B=1, lo=777, hi=777, Hq=32, Hk=8, D=128, page=16, fmt="bf16", window=0),
        # 256 sequences of mixed lengths over an 8-bit cache: a serving batch
        dict(name="attention_256_fp8", op="attention", B=256, lo=1, hi=4096, Hq=32, Hk=8, D=128, page=64, fmt="fp8", window=0),
        # one long document: the length is what there is to split
        dict(name="attention_1x131072", op="attention", B=1, lo=131072, hi=131072, Hq=32, Hk=4, D=128, page=64, fmt="bf16", window=0),
        # wide heads, a ragged batch with an idle place in it
        dict(name="attention_64_d256", op="attention", B=64, lo=0, hi=8192, Hq=16, Hk=2, D=256, page=32, fmt="bf16", window=0),
        # a sliding window over long sequences, a key head for every query head, pages of 24
        dict(name="attention_48_window", op="attention", B=48, lo=100, hi=16384, Hq=16, Hk=16, D=64, page=24, fmt="bf16", window=1024),
        # decode steps: a few sequences, and a batch
        dict(name="step_4", op="step", B=4, lo=64, hi=600, Hq=32, Hk=8, D=128, page=16, fmt="bf16", window=0),
        dict(name="step_64", op="step", B=64, lo=33, hi=4096, Hq=32, Hk=8, D=128, page=64, fmt="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "attention", "attention", "step"])
    D = rng.choice([64, 96, 128, 128, 192, 256])
    if op == "norm_rope":
        interleaved = rng.random() < 0.5
        R = rng.choice([r for r in (32, 64, D) if r <= D])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5])
        T = _log(rng, 1, max(1, min(32768, 32768 * 40 * 128 // (2 * (Hq + Hk) * D))))
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=R, start=rng.choice([0, D - R]), interleaved=interleaved,
                    x=rng.choice(["bf16", "f32"]), packed=rng.random() < 0.5)
    page = rng.choice([8, 16, 24, 32, 64, 128])
    fmt = rng.choice(["bf16", "fp8"])
    if op == "cache":
        Hk = rng.choice([1, 2, 5, 8])
        T = _log(rng, 1, max(1, min(32768, 32768 * 8 * 128 // (2 * Hk * D))))
        return dict(op=op, T=T, Hk=Hk, D=D, page=page, fmt=fmt, skip=rng.choice([0.0, 0.1]))
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8, 16])
    B = _log(rng, 1, 256)
    # no more cached values than 64 sequences of up to 4096 tokens with 4 heads of 256
    hi = _log(rng, 16, max(16, min(131072, 64 * 4096 * 4 * 256 // (B * Hk * D))))
    if op == "step":
        return dict(op=op, B=B, lo=max(1, hi // 16), hi=hi, Hq=Hq, Hk=Hk, D=D, page=page, fmt="bf16", window=0)
    window = rng.choice([0, 0, 128, 1000])
    return dict(op=op, B=B, lo=rng.choice([0, 1, hi // 7, hi]), hi=hi, Hq=Hq, Hk=Hk, D=D, page=page, fmt=fmt, window=window)


def _lens(case):
    """The batch's lengths: evenly spread over [lo, hi]; the seed decides only which sequence has which."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _attended(case):
    w = case["window"]
    return sum(min(n, w) if w else n for n in _lens(case))


def _row_bytes(case):
    return 2 * case["D"] if case["fmt"] == "bf16" else case["D"] + 4 * -(-case["D"] // 128)


def work(case):
    D = case["D"]
    if case["op"] == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": n * ((2 if case["x"] == "bf16" else 4) + 2) + case["T"] * 4 * (case["R"] + 1), "flops": 7 * n}
    if case["op"] == "cache":
        n = 2 * case["T"] * case["Hk"]
        return {"bytes": n * (2 * 2 * D + 2 * _row_bytes(case)) + 16 * case["T"], "flops": (6 if case["fmt"] == "fp8" else 0) * n * D}
    keys = _attended(case)
    got = {"bytes": 2 * keys * case["Hk"] * _row_bytes(case) + 4 * case["B"] * case["Hq"] * D + 4 * (keys // case["page"] + 2 * case["B"]),
           "flops": 4 * keys * case["Hq"] * D}
    if case["op"] == "step":
        got["bytes"] += case["B"] * (2 * case["Hk"] * (2 * D + _row_bytes(case)) + 4 * (D + 4))
    return got


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _angles(positions, R):
    """The rotation table a program keeps: fp32 [positions, R], cosines and then sines."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _encode(x):
    """fp32 [..., D] -> e4m3 codes uint8 [..., D] and scale bytes uint8 [..., 4 * ceil(D / 128)] (unused bytes 127)."""
    D = x.shape[-1]
    b = x.unflatten(-1, (D // 32, 32))
    amax = b.abs().amax(-1)
    f, ex = torch.frexp(amax)
    e = torch.where(f <= 0.875, ex - 9, ex - 8).clamp(-126, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
    scales = torch.full((*x.shape[:-1], 4 * -(-D // 128)), 127, dtype=torch.uint8, device=x.device)
    scales[..., :D // 32] = (e + 127).to(torch.uint8)
    return codes, scales


def _decode(codes, scales):
    """The fp32 values that codes and scale bytes stand for."""
    D = codes.shape[-1]
    s = (scales[..., :D // 32].to(torch.int32) << 23).view(torch.float32)
    return (codes.view(torch.float8_e4m3fn).float().unflatten(-1, (D // 32, 32)) * s.unsqueeze(-1)).flatten(-2)


def _cache(case, pages, g=None):
    """A paged cache [pages, Hk, page, D], empty or filled with rows of normal values."""
    shape = (pages, case["Hk"], case["page"], case["D"])
    st = {}
    for n in ("k", "v"):
        if case["fmt"] == "bf16":
            st[n] = _randn(g, shape, torch.bfloat16) if g is not None else torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
            st[n + "_scales"] = None
        elif g is not None:
            st[n], st[n + "_scales"] = _encode(_randn(g, shape))
        else:
            st[n] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            st[n + "_scales"] = torch.full((*shape[:3], 4 * -(-case["D"] // 128)), 127, dtype=torch.uint8, device=DEV)
    return st


def _pages(case, lens, rng, room):
    """Pages of every sequence at random places of the pool, -1 where a sequence has none. `room`: sequences start with a page."""
    need = [max(-(-n // case["page"]), room) for n in lens]
    places = rng.permutation(sum(need) + 3)
    table = np.full((case["B"], max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = places[at:at + n]
        at += n
    return table, sum(need) + 3


def _norm_rope_inputs(case, g, n, positions):
    D, dt = case["D"], torch.bfloat16 if case.get("x", "bf16") == "bf16" else torch.float32
    Hq, Hk = case["Hq"], case["Hk"]
    if case.get("packed"):
        rows = _randn(g, (n, (Hq + 2 * Hk) * D), dt, 2.0).view(n, Hq + 2 * Hk, D)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    else:
        q, k, v = (_randn(g, (n, h, D), dt, 2.0) for h in (Hq, Hk, Hk))
    return dict(q=q, k=k, v=v, positions=positions, q_weight=(1.0 + _randn(g, (D,), std=0.1)).bfloat16(),
                k_weight=(1.0 + _randn(g, (D,), std=0.1)).bfloat16())


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    op, D = case["op"], case["D"]
    st = {"case": case}
    if op == "norm_rope":
        # prompts of up to 4096 tokens one after another
        first = int(rng.integers(0, 1000))
        positions = (torch.arange(case["T"], device=DEV) % 4096 + first).to(torch.int32)
        st |= _norm_rope_inputs(case, g, case["T"], positions)
        st["table"] = _angles(8192, case["R"])
    elif op == "cache":
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        st |= _cache(case, pages)
        # rows as a norm and a projection give them: keys of unit size, values of a spread of sizes
        st["new_k"] = _randn(g, (T, case["Hk"], D), torch.bfloat16)
        st["new_v"] = (_randn(g, (T, case["Hk"], D)) * torch.exp2(_randn(g, (T, case["Hk"], 1), std=2.0))).bfloat16()
        place = rng.permutation(pages)[np.arange(T) // page].astype(np.int64) * page + np.arange(T) % page
        write = place.copy()
        write[rng.random(T) < case["skip"]] = -1
        st["slots"] = torch.from_numpy(write).to(DEV)         # the padded tokens are written nowhere,
        st["read_slots"] = torch.from_numpy(write).to(DEV)    # and read as zero
    else:
        lens = rng.permutation(_lens(case)).tolist()
        table, pages = _pages(case, lens, rng, 1 if op == "step" else 0)
        st |= _cache(case, pages, g)
        st["block_table"] = torch.from_numpy(table).to(DEV)
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["span"] = max(max(min(n, case["window"]) if case["window"] else n for n in lens), 1)
        st["scale"] = 1.0 / math.sqrt(D)
        if op == "attention":
            st["q"] = _randn(g, (case["B"], case["Hq"], D), torch.bfloat16, 1.5)
            if case["fmt"] == "bf16":  # what lies behind a sequence's last key is not defined
                page = case["page"]
                ends = [(int(table[b, n // page]), n % page) for b, n in enumerate(lens) if n % page]
                if ends:
                    p, at = (torch.tensor(x, device=DEV) for x in zip(*ends))
                    tail = (torch.arange(page, device=DEV)[None, :] >= at[:, None])[:, None, :, None]
                    for n in ("k", "v"):
                        st[n][p] = torch.where(tail, torch.nan, st[n][p])
        else:
            st |= {n: x for n, x in _norm_rope_inputs(case, g, case["B"], st["seq_lens"] - 1).items() if n not in ("k", "v")} | \
                {"new_" + n: _randn(g, (case["B"], case["Hk"], D), torch.bfloat16, 2.0) for n in ("k", "v")}
            st["table"] = _angles(case["hi"], D)
            page = case["page"]
            st["slots"] = torch.tensor([int(table[b, (n - 1) // page]) * page + (n - 1) % page for b, n in enumerate(lens)],
                                       dtype=torch.int64, device=DEV)
    if own:
        _keep(st)
    return st


def _keep(st):
    """What a program keeps beside its tensors: the cache's handle, the marshalled calls on its buffers, their workspace."""
    import engram_gram_hash_02_gb300 as E
    case = st["case"]
    D, T = case["D"], case.get("T", case.get("B"))
    if "table" in st:
        nr = E.NormRope(st["q_weight"], st["k_weight"], EPS, st["table"], start=case.get("start", 0),
                        interleaved=case.get("interleaved", False))
    if case["op"] == "norm_rope":
        st["q_out"], st["k_out"] = (torch.empty((T, case[h], D), dtype=torch.bfloat16, device=DEV) for h in ("Hq", "Hk"))
        st["plan"] = E.QKNormRopePlan(nr, st["q"], st["k"], st["positions"], q_out=st["q_out"], k_out=st["k_out"])
        return
    cache = E.KVCache(st["k"], st["v"], st["k_scales"], st["v_scales"])
    if case["op"] == "cache":
        st["k_out"], st["v_out"] = (torch.empty((T, case["Hk"], D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        st["plan"] = E.KVWritePlan(cache, st["new_k"], st["new_v"], st["slots"])
        st["read"] = E.KVReadPlan(cache, st["read_slots"], k_out=st["k_out"], v_out=st["v_out"])
        return
    st["out"] = torch.empty((T, case["Hq"], D), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "attention":
        st["lse"] = torch.empty((T, case["Hq"]), dtype=torch.float32, device=DEV)
        st["plan"] = E.PagedAttentionPlan(cache, st["q"], st["block_table"], st["seq_lens"], scale=st["scale"], window=case["window"],
                                          out=st["out"], lse=st["lse"])
    else:
        st["plan"] = E.AttentionStepPlan(nr, cache, st["q"], st["new_k"], st["new_v"], st["positions"], st["slots"],
                                         st["block_table"], st["seq_lens"], scale=st["scale"], window=case["window"], out=st["out"])


# ------------------------------------------------------------------------------------------------ one pass

def _norm_rope(x, w, table, positions, start, interleaved):
    """fp32 [T, heads, D]: RMS norm over D, weight, rotation of D's part [start, start + R)."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    R = table.shape[1]
    c, s = table[positions.long()].unsqueeze(1).chunk(2, -1)
    r = y[..., start:start + R]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r.chunk(2, -1)
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y[..., :start], r, y[..., start + R:]], -1)


def _write(st, n, rows, slots):
    """rows fp32 [T, Hk, D] to their slots of the cache; slots below 0 are skipped."""
    page = st["case"]["page"]
    keep = slots >= 0
    p, at = slots[keep] // page, slots[keep] % page
    if st["case"]["fmt"] == "bf16":
        st[n][p, :, at] = rows[keep].bfloat16()
    else:
        st[n][p, :, at], st[n + "_scales"][p, :, at] = _encode(rows[keep])


def _rows(st, n, p, at):
    """fp32 rows [..., Hk, D] of the cache at pages p and places at."""
    x = st[n][p, :, at]
    return x.float() if st["case"]["fmt"] == "bf16" else _decode(x, st[n + "_scales"][p, :, at])


def _attend(st, q):
    case = st["case"]
    B, Hq, D = q.shape
    lens = st["seq_lens"].long()
    first = (lens - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
    pos = first[:, None] + torch.arange(st["span"], device=DEV)                     # [B, S]
    there = pos < lens[:, None]
    pos = torch.where(there, pos, torch.zeros_like(pos))
    p = torch.gather(st["block_table"], 1, pos // case["page"]).long().clamp(min=0)
    at = pos % case["page"]
    hide = ~there[:, :, None, None]
    k = _rows(st, "k", p, at).masked_fill(hide, 0.0)                                # [B, S, Hk, D]
    v = _rows(st, "v", p, at).masked_fill(hide, 0.0)
    qg = q.float().view(B, case["Hk"], Hq // case["Hk"], D) * st["scale"]
    s = torch.matmul(qg, k.permute(0, 2, 3, 1))                                     # [B, Hk, G, S]
    s = s.masked_fill(~there[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(B, Hq, D).bfloat16(), (m + torch.log(total)).reshape(B, Hq)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        st["plan"].run()
        if op == "norm_rope":
            return st["q_out"], st["k_out"]
        if op == "cache":
            st["read"].run()
            return st["k_out"], st["v_out"]
        return (st["out"], st["lse"]) if op == "attention" else (st["out"], st["k"], st["v"])
    if op == "norm_rope":
        how = (st["table"], st["positions"], case["start"], case["interleaved"])
        return _norm_rope(st["q"], st["q_weight"], *how).bfloat16(), _norm_rope(st["k"], st["k_weight"], *how).bfloat16()
    if op == "cache":
        _write(st, "k", st["new_k"].float(), st["slots"])
        _write(st, "v", st["new_v"].float(), st["slots"])
        slots = st["read_slots"]
        there = (slots >= 0)[:, None, None]
        p, at = slots.clamp(min=0) // case["page"], slots.clamp(min=0) % case["page"]
        return tuple(_rows(st, n, p, at).masked_fill(~there, 0.0).bfloat16() for n in ("k", "v"))
    if op == "attention":
        return _attend(st, st["q"])
    how = (st["table"], st["positions"], 0, False)
    _write(st, "k", _norm_rope(st["new_k"], st["k_weight"], *how), st["slots"])
    _write(st, "v", st["new_v"].float(), st["slots"])
    return _attend(st, _norm_rope(st["q"], st["q_weight"], *how))[0], st["k"], st["v"]


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_turn(x, w, table, positions, start, interleaved):
    """Norm and rotation as complex numbers."""
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    half = table.shape[1] // 2
    turn = torch.complex(table[:, :half].double(), table[:, half:].double())[positions.long()][:, None, :]
    i = torch.arange(half, device=DEV)
    ia, ib = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + half + i)
    z = torch.complex(y[..., ia], y[..., ib]) * turn
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _exact_fp8(x):
    """The values that blocks of 32 stand for after the smallest power of two that brings them to 448 or less, and rounding to
    three bits behind the leading one (steps of 2^-9 at the least), ties to even."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    e = torch.where(top * torch.exp2(-e) > 448.0, e + 1, e)
    e = torch.where(top * torch.exp2(1 - e) <= 448.0, e - 1, e).clamp(min=-126)
    e = torch.where(top > 0, e, torch.zeros_like(e))
    u = b * torch.exp2(-e)
    lead = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(lead - 3)
    return (torch.round(u / step) * step * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    op, page = case["op"], case.get("page")
    if op == "norm_rope":
        how = (st["table"], st["positions"], case["start"], case["interleaved"])
        return _exact_turn(st["q"], st["q_weight"], *how), _exact_turn(st["k"], st["k_weight"], *how)
    if op == "cache":
        there = (st["slots"] >= 0).double()[:, None, None]
        return tuple((x.double() if case["fmt"] == "bf16" else _exact_fp8(x)) * there for x in (st["new_k"], st["new_v"]))
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    q, new = st["q"].double(), {}
    if op == "step":
        how = (st["table"], st["positions"], 0, False)
        q = _exact_turn(st["q"], st["q_weight"], *how)
        new = {"k": _exact_turn(st["new_k"], st["k_weight"], *how), "v": st["new_v"].double()}
    out, lse = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV), torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["seq_lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        pg = st["block_table"][b, :-(-n // page)].long()
        kv = []
        for name in ("k", "v"):
            x = st[name][pg].transpose(1, 2).flatten(0, 1)[lo:n]                    # [n - lo, Hk, D]
            if case["fmt"] == "fp8":
                byte = st[name + "_scales"][pg].transpose(1, 2).flatten(0, 1)[lo:n, :, :D // 32].double()
                x = x.view(torch.float8_e4m3fn).to(torch.float64) * torch.exp2(byte - 127).repeat_interleave(32, -1)
            x = x.double()
            if new:
                x[-1] = new[name][b].bfloat16()
            kv.append(x)
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            s = q[b, heads] @ kv[0][:, h].T * st["scale"]
            lse[b, heads] = torch.logsumexp(s, -1)
            out[b, heads] = torch.softmax(s, -1) @ kv[1][:, h]
    if op == "attention":
        return out, lse
    caches = []
    for name in ("k", "v"):
        c = st[name].double()
        c[st["slots"] // page, :, st["slots"] % page] = new[name]
        caches.append(c)
    return out, caches[0], caches[1]
