"""More attention operators of a decoder layer, in their plain form and through the package's entry points.

Three operators over one paged key-value cache (bf16, or 8-bit with one power-of-two scale per 32 values):
`prompt` (all new tokens of ragged sequences: causal, a window, documents, a prefix that is seen both ways), `token` (one new token
per sequence) and `shared` (one new token per sequence, groups of sequences that share a prefix). Their scores may be capped
(cap * tanh(s / cap)) and carry a bias that falls with distance (-slope * |p - j|).
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a short question, the first prompt of a conversation: latency
        dict(name="prompt_1x37", op="prompt", B=1, new_lo=37, new_hi=37, old=0, Hq=32, Hk=8, D=128, page=16, fmt="bf16", window=0,
             docs=0, prefix=False, cap=0.0, slopes=False),
        # drafted tokens checked in one pass: five new tokens for each of 32 sequences
        dict(name="prompt_32x5", op="prompt", B=32, new_lo=5, new_hi=5, old=4096, Hq=32, Hk=8, D=128, page=64, fmt="bf16", window=0,
             docs=0, prefix=False, cap=0.0, slopes=False),
        # eight prompts of 4096 tokens at once
        dict(name="prompt_8x4096", op="prompt", B=8, new_lo=4096, new_hi=4096, old=0, Hq=32, Hk=8, D=128, page=64, fmt="bf16",
             window=0, docs=0, prefix=False, cap=0.0, slopes=False),
        # documents packed into one sequence, wide heads, capped scores
        dict(name="prompt_docs_cap", op="prompt", B=1, new_lo=16384, new_hi=16384, old=0, Hq=16, Hk=2, D=256, page=32, fmt="bf16",
             window=0, docs=1500, prefix=False, cap=50.0, slopes=False),
        # a chunk of 512 tokens of each of 16 long prompts over what is cached of them in 8 bits, with a sliding window
        dict(name="prompt_16x512_fp8", op="prompt", B=16, new_lo=512, new_hi=512, old=8192, Hq=32, Hk=8, D=128, page=64, fmt="fp8",
             window=4096, docs=0, prefix=False, cap=0.0, slopes=False),
        # prompts of odd lengths whose beginning is seen both ways, distance bias, a key head for every query head, pages of 24
        dict(name="prompt_7_prefix_slopes", op="prompt", B=7, new_lo=113, new_hi=2011, old=0, Hq=12, Hk=12, D=64, page=24, fmt="bf16",
             window=0, docs=0, prefix=True, cap=0.0, slopes=True),
        # a single decode of a model with capped scores: latency
        dict(name="token_1x777_cap", op="token", B=1, lo=777, hi=777, Hq=32, Hk=8, D=128, page=16, fmt="bf16", window=0, cap=50.0,
             slopes=False),
        # wide heads with capped scores, a ragged batch with an idle place in it
        dict(name="token_64_cap_d256", op="token", B=64, lo=0, hi=8192, Hq=16, Hk=2, D=256, page=32, fmt="bf16", window=0, cap=30.0,
             slopes=False),
        # a serving batch of a model with a distance bias over an 8-bit cache
        dict(name="token_128_slopes_fp8", op="token", B=128, lo=1, hi=4096, Hq=32, Hk=8, D=128, page=64, fmt="fp8", window=0, cap=0.0,
             slopes=True),
        # four answers drawn from one short prompt
        dict(name="shared_4x500", op="shared", groups="4", prefix_lo=500, prefix_hi=500, lo=1, hi=64, Hq=32, Hk=8, D=128, page=16,
             fmt="bf16", cap=0.0, slopes=False),
        # 128 questions about one long document
        dict(name="shared_128x16384", op="shared", groups="128", prefix_lo=16384, prefix_hi=16384, lo=16, hi=1024, Hq=32, Hk=8, D=128,
             page=64, fmt="bf16", cap=0.0, slopes=False),
        # groups of different sizes with a system prompt each, capped scores over an 8-bit cache
        dict(name="shared_6_groups_fp8", op="shared", groups="40+24+17+9+5+1", prefix_lo=2048, prefix_hi=8191, lo=0, hi=700,
             Hq=32, Hk=4, D=128, page=16, fmt="fp8", cap=30.0, slopes=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "token", "shared"])
    D = rng.choice([64, 96, 128, 128, 192, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    fmt = rng.choice(["bf16", "fp8"])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, Hq=Hq, Hk=Hk, D=D, page=page, fmt=fmt, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                slopes=rng.random() < 0.3)
    if op == "prompt":
        # no more than eight prompts of 4096 tokens with 32 heads of 128 compute
        room = 8 * 4096 * 4096 * 32 * 128 // (Hq * D)
        B = _log(rng, 1, 32)
        new = _log(rng, 1, max(1, min(8192, math.isqrt(room // B))))
        old = rng.choice([0, 0, _log(rng, 1, 8192)])
        old = min(old, max(0, room // (B * new) - new), 2 ** 27 // (B * Hk * D))
        docs = rng.choice([0, 0, max(1, new // 5)])
        case |= dict(B=B, new_lo=max(1, new // rng.choice([1, 3])), new_hi=new, old=old, docs=docs,
                     window=rng.choice([0, 0, 0, 100, 1000]), prefix=docs == 0 and rng.random() < 0.3)
        return case
    if op == "token":
        B = _log(rng, 1, 256)
        # no more cached values than 64 sequences of up to 4096 tokens with 4 heads of 256
        hi = _log(rng, 16, max(16, min(131072, 64 * 4096 * 4 * 256 // (B * Hk * D))))
        case |= dict(B=B, lo=rng.choice([0, 1, hi // 7, hi]), hi=hi, window=rng.choice([0, 0, 1000]))
        return case
    groups = [_log(rng, 1, 64) for _ in range(rng.choice([1, 1, 2, 5]))]
    B = sum(groups)
    longest = _log(rng, 16, max(16, min(32768, 16384 * 128 * 32 * 128 // (B * Hq * D))))
    hi = _log(rng, 1, max(1, min(1024, 2 ** 27 // (B * Hk * D))))
    case |= dict(groups="+".join(map(str, groups)), prefix_lo=rng.choice([0, longest // 3, longest]), prefix_hi=longest, lo=rng.choice([0, 1, hi]), hi=hi)
    return case


def _spread(n, lo, hi):
    """n lengths evenly spread over [lo, hi]; the seed decides only which sequence has which."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _groups(case):
    """The sizes of a batch's groups."""
    return [int(n) for n in case["groups"].split("+")]


def _row_bytes(case):
    return 2 * case["D"] if case["fmt"] == "bf16" else case["D"] + 4 * -(-case["D"] // 128)


def _new(case):
    return _spread(case["B"], case["new_lo"], case["new_hi"])


def _old(case):
    """Tokens cached before the new ones, per sequence: evenly spread up to the case's number."""
    return _spread(case["B"], case["old"] // 4, case["old"]) if case["old"] else [0] * case["B"]


def _doc_starts(case, p, shift=0):
    """The first positions of the documents that positions p lie in: lengths from a sixteenth of the case's to twice it, in an
    irregular order; `shift` tokens of the first one are gone."""
    lengths = np.maximum(case["docs"] * (1 + 3 * (np.arange(11) * 7 % 11)) // 16, 1)
    bounds = np.concatenate([[0], np.cumsum(np.tile(lengths, int(p[-1] + shift) // int(lengths.sum()) + 1))])
    return np.maximum(bounds[np.searchsorted(bounds, p + shift, side="right") - 1] - shift, 0)


def _visible(case, n, old):
    """Pairs (query, key) that a prompt of n new tokens over `old` cached ones has, and the keys that any of them sees (the prefix
    seen both ways is a quarter of the new tokens)."""
    p = old + np.arange(n, dtype=np.int64)
    lo = np.zeros(n, np.int64)
    if case["window"]:
        lo = np.maximum(lo, p + 1 - case["window"])
    if case["docs"]:
        lo = np.maximum(lo, _doc_starts(case, p))
    hi = p + 1
    if case["prefix"]:
        hi = np.maximum(hi, old + n // 4)
    return int((hi - lo).sum()), int(old + n - lo.min())


def work(case):
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    row = 2 * Hk * _row_bytes(case)
    if case["op"] == "prompt":
        new, old = _new(case), _old(case)
        seen = [_visible(case, n, o) for n, o in zip(new, old)]
        T, pairs, keys = sum(new), sum(s[0] for s in seen), sum(s[1] for s in seen)
        entries = keys // case["page"] + 2 * case["B"]
    elif case["op"] == "token":
        lens = _spread(case["B"], case["lo"], case["hi"])
        T, pairs = case["B"], sum(min(n, case["window"]) if case["window"] else n for n in lens)
        keys, entries = pairs, pairs // case["page"] + 2 * case["B"]
    else:
        sizes = _groups(case)
        T, G = sum(sizes), len(sizes)
        lens, prefixes = _spread(T, case["lo"], case["hi"]), _spread(G, case["prefix_lo"], case["prefix_hi"])
        pairs = sum(lens) + sum(n * g for n, g in zip(prefixes, sizes))
        keys = sum(lens) + sum(prefixes)
        entries = keys // case["page"] + 2 * (T + G)
    return {"bytes": keys * row + T * Hq * (4 * D + 4) + 4 * entries, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _encode(x):
    """fp32 [..., D] -> e4m3 codes uint8 [..., D] and scale bytes uint8 [..., 4 * ceil(D / 128)] (unused bytes 127): per block of 32
    the smallest power of two that brings it to 448 or less."""
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


def _cache(case, pages, g):
    """A paged cache [pages, Hk, page, D] filled with rows of normal values."""
    shape = (pages, case["Hk"], case["page"], case["D"])
    st = {}
    for n in ("k", "v"):
        st[n], st[n + "_scales"] = (_randn(g, shape, torch.bfloat16), None) if case["fmt"] == "bf16" else _encode(_randn(g, shape))
    return st


def _table(lens, page, rng, places):
    """int32 [len(lens), width]: pages of every sequence, taken from `places`; -1 where a sequence has none."""
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [next(places) for _ in range(n)]
    return table


def _undefined_tails(st, case, table, lens):
    """What lies behind a sequence's last key is not defined."""
    page = case["page"]
    ends = [(int(table[b, n // page]), n % page) for b, n in enumerate(lens) if n % page]
    if not ends:
        return
    p, at = (torch.tensor(x, device=DEV) for x in zip(*ends))
    tail = (torch.arange(page, device=DEV)[None, :] >= at[:, None])[:, None, :, None]
    for n in ("k", "v"):
        junk = torch.nan if case["fmt"] == "bf16" else 0x7F
        st[n][p] = torch.where(tail, torch.full((), junk, dtype=st[n].dtype, device=DEV), st[n][p])


def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    op, D, Hq, page = case["op"], case["D"], case["Hq"], case["page"]
    st = {"case": case, "scale": 1.0 / math.sqrt(D)}
    prefixes = []
    if op == "prompt":
        order = rng.permutation(case["B"])
        new = [_new(case)[i] for i in order]
        old = [_old(case)[i] for i in rng.permutation(case["B"])]
        lens = [n + o for n, o in zip(new, old)]
        st["new"], T = new, sum(new)
        st["cu_seqlens"] = _dev([0, *np.cumsum(new).tolist()])
        if case["docs"]:
            st["doc_starts"] = _dev(np.concatenate([_doc_starts(case, np.arange(n - m, n), int(rng.integers(0, case["docs"])))
                                                    for n, m in zip(lens, new)]))
        if case["prefix"]:                                    # the first quarter of the new tokens sees all of itself
            st["prefix_ends"] = _dev(np.concatenate([np.full(m, n - m + m // 4) for n, m in zip(lens, new)]))
    elif op == "token":
        lens, T = [_spread(case["B"], case["lo"], case["hi"])[i] for i in rng.permutation(case["B"])], case["B"]
    else:
        sizes = _groups(case)
        T = sum(sizes)
        lens = [_spread(T, case["lo"], case["hi"])[i] for i in rng.permutation(T)]
        prefixes = _spread(len(sizes), case["prefix_lo"], case["prefix_hi"])
        st["groups"] = _dev([0, *np.cumsum(sizes).tolist()])
    pages = sum(-(-n // page) for n in [*lens, *prefixes]) + 3
    places = iter(rng.permutation(pages).tolist())
    st |= _cache(case, pages, g)
    table = _table(lens, page, rng, places)
    _undefined_tails(st, case, table, lens)
    st["lens"], st["seq_lens"], st["block_table"] = lens, _dev(lens), torch.from_numpy(table).to(DEV)
    if op == "shared":
        table = _table(prefixes, page, rng, places)
        _undefined_tails(st, case, table, prefixes)
        st["prefixes"], st["prefix_lens"], st["prefix_table"] = prefixes, _dev(prefixes), torch.from_numpy(table).to(DEV)
    # scores of a spread of 1.5, and where they are capped of a third of the cap
    st["q"] = _randn(g, (T, Hq, D), torch.bfloat16, case["cap"] / 3 if case["cap"] else 1.5)
    # slopes 2^(-8 (h + 1) / Hq), as models with a distance bias have them
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq).float() if case["slopes"] else None
    if own:
        _keep(st)
    return st


def _keep(st):
    """What a program keeps beside its tensors: the cache's handle, the marshalled call on its buffers, its workspace."""
    import engram_gram_hash_02_gb300 as E
    case = st["case"]
    cache = E.KVCache(st["k"], st["v"], st["k_scales"], st["v_scales"])
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    how = dict(scale=st["scale"], out=st["out"], lse=st["lse"], cap=case["cap"], slopes=st["slopes"])
    if case["op"] == "prompt":
        st["plan"] = E.PromptAttentionPlan(cache, st["q"], st["cu_seqlens"], st["block_table"], st["seq_lens"], window=case["window"],
                                           doc_starts=st.get("doc_starts"), prefix_ends=st.get("prefix_ends"), **how)
    elif case["op"] == "token":
        st["plan"] = E.PagedAttentionPlan(cache, st["q"], st["block_table"], st["seq_lens"], window=case["window"], **how)
    else:
        st["plan"] = E.SharedAttentionPlan(cache, st["q"], st["prefix_table"], st["prefix_lens"], st["groups"], st["block_table"],
                                           st["seq_lens"], **how)


# ------------------------------------------------------------------------------------------------ one pass

def _rows(st, table, b, n):
    """fp32 keys and values [n, Hk, D] of the n tokens in row b of a page table."""
    case = st["case"]
    pos = torch.arange(n, device=DEV)
    p, at = table[b].index_select(0, pos // case["page"]).long(), pos % case["page"]
    got = []
    for name in ("k", "v"):
        x = st[name][p, :, at]
        if case["fmt"] == "bf16":
            got.append(x.float())
        else:
            s = (st[name + "_scales"][p, :, at][..., :case["D"] // 32].to(torch.int32) << 23).view(torch.float32)
            got.append((x.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2))
    return got


def _attend(st, q, k, v, p, lo, hi):
    """Rows q fp32 [n, Hq, D] at positions p [n] over the keys [lo, hi) of k and v [L, Hk, D]: (out, lse) in 32 bits."""
    case = st["case"]
    n, Hq, D = q.shape
    L, Hk = k.shape[:2]
    out, lse = torch.zeros((n, Hq, D), device=DEV), torch.full((n, Hq), -math.inf, device=DEV)
    if L == 0:
        return out, lse
    j = torch.arange(L, device=DEV)
    step = max(1, 2 ** 28 // (Hq // Hk * L))                  # rows at a time
    for a in range(0, n, step):
        rows = slice(a, min(n, a + step))
        hide = (j < lo[rows, None]) | (j >= hi[rows, None])                                  # [r, L]
        far = (p[rows, None] - j).abs().float() if st["slopes"] is not None else None
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            s = torch.matmul(q[rows, heads].transpose(0, 1) * st["scale"], k[:, h].T)        # [G, r, L]
            if case["cap"]:
                s = torch.tanh(s / case["cap"]) * case["cap"]
            if far is not None:
                s = s - st["slopes"][heads, None, None] * far
            s = s.masked_fill(hide, -math.inf)
            m = s.amax(-1, keepdim=True)
            e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
            total = e.sum(-1, keepdim=True)
            o = torch.matmul(e, v[:, h]) / torch.where(total == 0, torch.ones_like(total), total)
            out[rows, heads] = o.transpose(0, 1)
            lse[rows, heads] = (m + torch.log(total)).squeeze(-1).T
    return out, lse


def _interval(st, t0, n, length):
    """Positions and visible keys [lo, hi) of the n new tokens of a prompt that ends at `length`; t0: its first row."""
    case = st["case"]
    p = torch.arange(length - n, length, device=DEV)
    lo, hi = torch.zeros_like(p), p + 1
    if case["window"]:
        lo = torch.maximum(lo, p + 1 - case["window"])
    if "doc_starts" in st:
        lo = torch.maximum(lo, st["doc_starts"][t0:t0 + n].long())
    if "prefix_ends" in st:
        hi = torch.maximum(hi, st["prefix_ends"][t0:t0 + n].long())
    return p, lo, hi


def run(st):
    if own:
        st["plan"].run()
        return st["out"], st["lse"]
    case, q = st["case"], st["q"].float()
    outs = []
    if case["op"] == "prompt":
        t0 = 0
        for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
            outs.append(_attend(st, q[t0:t0 + n], *_rows(st, st["block_table"], b, length), *_interval(st, t0, n, length)))
            t0 += n
    else:
        group, prefix = -1, None
        ends = np.cumsum(_groups(case)) if case["op"] == "shared" else None
        for b, n in enumerate(st["lens"]):
            k, v = _rows(st, st["block_table"], b, n)
            first = max(0, n - case["window"]) if case.get("window") else 0
            if ends is not None:
                g = int(np.searchsorted(ends, b, side="right"))
                if g != group:
                    group, prefix = g, _rows(st, st["prefix_table"], g, st["prefixes"][g])
                k, v = (torch.cat(x) for x in zip(prefix, (k, v)))
            L = k.shape[0]
            at = torch.arange(1, device=DEV)
            outs.append(_attend(st, q[b:b + 1], k, v, at + (L - 1), at + first, at + L))
    return torch.cat([o for o, _ in outs]).bfloat16(), torch.cat([x for _, x in outs])


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_rows(st, name, table, b, n):
    """The 64-bit rows [n, Hk, D] of a sequence, page by page."""
    case, page = st["case"], st["case"]["page"]
    pages = table[b, :-(-n // page)].long()
    x = st[name][pages].transpose(1, 2).flatten(0, 1)[:n]
    if case["fmt"] == "bf16":
        return x.double()
    byte = st[name + "_scales"][pages].transpose(1, 2).flatten(0, 1)[:n, :, :case["D"] // 32].double()
    return x.view(torch.float8_e4m3fn).double() * torch.exp2(byte - 127).repeat_interleave(32, -1)


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    Hq, Hk, D, cap, slopes = case["Hq"], case["Hk"], case["D"], case["cap"], st["slopes"]
    T = st["q"].shape[0]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    new = st["new"] if case["op"] == "prompt" else [1] * T
    t0 = 0
    for b, (n, length) in enumerate(zip(new, st["lens"])):
        k, v = (_exact_rows(st, x, st["block_table"], b, length) for x in ("k", "v"))
        if case["op"] == "shared":
            g = sum(b >= e for e in np.cumsum(_groups(case)).tolist())
            k, v = (torch.cat([_exact_rows(st, x, st["prefix_table"], g, st["prefixes"][g]), y]) for x, y in (("k", k), ("v", v)))
        L = k.shape[0]
        if L:
            rows = 4096
            for a in range(0, n, rows):
                r = min(rows, n - a)
                pos = torch.arange(L - n + a, L - n + a + r, device=DEV, dtype=torch.float64)[:, None]
                key = torch.arange(L, device=DEV, dtype=torch.float64)[None, :]
                seen = key <= pos
                if case["op"] == "prompt" and case["prefix"]:
                    seen |= key < st["prefix_ends"][t0 + a:t0 + a + r, None]
                if case["op"] == "prompt" and case["docs"]:
                    seen &= key >= st["doc_starts"][t0 + a:t0 + a + r, None]
                if case.get("window"):
                    seen &= key > pos - case["window"]
                for h in range(Hq):
                    s = st["q"][t0 + a:t0 + a + r, h].double() @ k[:, h * Hk // Hq].T / math.sqrt(D)
                    if cap:
                        s = cap * torch.tanh(s / cap)
                    if slopes is not None:
                        s -= float(slopes[h]) * (pos - key).abs()
                    s.masked_fill_(~seen, -math.inf)
                    lse[t0 + a:t0 + a + r, h] = torch.logsumexp(s, -1)
                    out[t0 + a:t0 + a + r, h] = torch.softmax(s, -1).nan_to_num(0.0) @ v[:, h * Hk // Hq]
        t0 += n
    return out, lse
