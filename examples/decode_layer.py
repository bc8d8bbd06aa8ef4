"""A decoder layer served: its Engram residual, its attention over a paged cache, greedy decoding.

    python examples/decode_layer.py [--cache fp8] [--steps 24]

Three prompts of different lengths go through the layer at once: engram_forward adds the Engram residual to
the hyper-connection streams, a projection of their mean gives queries, keys and values (packed rows, fp32),
engram_qk_norm_rope norms and turns them, engram_kv_write fills the cache, and engram_paged_attention answers
for each prompt's last token. Then every step feeds back one token per sequence: engram_forward with the
previous tokens as lookback, and engram_attention_step (norm, rotation, cache write and attention in one call).
At the end the whole sequences go through once more as prompts, and the logits are compared.

Weights are random and the projections are the caller's own (plain torch): only the layer's plumbing is shown.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import engram_gram_hash_02_gb300 as E  # noqa: E402
from engram_synth import gen, get_workload  # noqa: E402
from engram_synth.case import make_tables, to_device  # noqa: E402

DEV = "cuda"
Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 8, 2, 64, 16


class Layer:
    """The weights of one layer: an Engram table and gate, packed qkv rows, head norms, an output head."""

    def __init__(self, w, seed: int):
        primes, offsets, rows = E.engram_layout(w.vocab_size, 1, w.max_ngram, w.n_heads)
        self.w, self.map = w, gen.batch_inputs(w)["token_map"]
        self.dims = E.make_dims(1, w.max_ngram, w.n_heads, w.head_dim, w.hidden, w.hc, w.raw_vocab, w.compressed_vocab,
                                int(self.map[w.pad_token_id]), w.eps, w.clamp)
        mult = E.hash_multipliers(w.layer_ids, w.max_ngram, w.compressed_vocab)
        self.tables = E.HashTables(*(to_device(x, DEV) for x in (self.map, mult, primes, offsets)))
        t = make_tables(w, rows, DEV, seed)[0]
        q, k = gen.gate_weights(w.hc, w.hidden, w.qk_std, seed, DEV)
        self.engram = E.LayerWeights(t["fmt"], t["table"], t["scales"], t["num_rows"],
                                     gen.wkv_weight(w.N, w.K, 0.5, seed, DEV), q, k)
        g = torch.Generator(device=DEV).manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.embedding = randn(w.raw_vocab, w.hidden)
        self.qkv = randn(w.hidden, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM) * w.hidden ** -0.5
        self.head = randn(Q_HEADS * HEAD_DIM + w.hidden, w.raw_vocab) * w.hidden ** -0.5
        weights = [(1 + 0.1 * randn(HEAD_DIM)).bfloat16() for _ in range(2)]
        self.nr = E.NormRope(*weights, w.eps, E.rope_table(4096, HEAD_DIM, device=DEV))

    def rows(self, ids, cu_seqlens, lookback=None):
        """Raw ids [T] -> the layer's input x [T, H] after its Engram residual, and its q, k, v rows (fp32 views)."""
        streams = self.embedding[ids.long()].unsqueeze(1).repeat(1, self.w.hc, 1)
        E.engram_forward(self.dims, self.tables, [self.engram], ids, [streams], cu_seqlens=cu_seqlens, lookback_ids=lookback)
        x = streams.mean(1)
        packed = (x @ self.qkv).view(len(ids), -1, HEAD_DIM)
        return x, packed.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)

    def logits(self, x, attended):
        return torch.cat([attended.float().flatten(1), x], 1) @ self.head


class Sequences:
    """The batch's paged cache: pages handed out one after another as sequences grow."""

    def __init__(self, batch: int, longest: int, fmt: str):
        width = -(-longest // PAGE)
        self.cache = E.KVCache.allocate(batch * width, PAGE, KV_HEADS, HEAD_DIM, fmt)
        # an engine takes pages from a pool as they are needed; here every sequence's are interleaved beforehand
        self.table = torch.arange(batch * width, dtype=torch.int32, device=DEV).view(width, batch).t().contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)

    def slots(self, seq, positions):
        page = self.table[seq.long(), positions.long() // PAGE].long()
        return page * PAGE + positions.long() % PAGE


def prompt(layer: Layer, seqs: Sequences, prompts: list) -> torch.Tensor:
    """The prompts through the layer at once; logits after each one's last token."""
    lens = [len(p) for p in prompts]
    ids = to_device(np.concatenate(prompts).astype(np.int32), DEV)
    cu = to_device(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), torch.tensor(lens, device=DEV))
    positions = (torch.arange(len(ids), device=DEV) - cu[seq]).to(torch.int32)
    x, (q, k, v) = layer.rows(ids, cu)
    turned_q, turned_k = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k, memory_format=torch.contiguous_format)
    E.engram_qk_norm_rope(layer.nr, q, k, positions, turned_q, turned_k)
    E.engram_kv_write(seqs.cache, turned_k, v, seqs.slots(seq, positions))
    seqs.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    last = cu[1:].long() - 1
    attended = E.engram_paged_attention(seqs.cache, turned_q[last], seqs.table, seqs.lens)
    return layer.logits(x[last], attended)


def decode(layer: Layer, seqs: Sequences, history: list, token: torch.Tensor, steps: int):
    """`steps` tokens per sequence, greedily; the logits after the last one. `history` grows."""
    B, n = len(history), layer.w.max_ngram - 1
    token_map = layer.tables.token_map
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    batch = torch.arange(B, device=DEV)
    lookback = torch.tensor([[-1] * max(0, n - len(h)) + [int(layer.map[t]) for t in h[-n:]] for h in history],
                            dtype=torch.int32, device=DEV)
    workspace = E.attention_workspace(seqs.cache, Q_HEADS, B)
    logits = None
    for _ in range(steps):
        x, (q, k, v) = layer.rows(token, cu, lookback)
        positions = seqs.lens.clone()                         # the new token's place
        seqs.lens += 1
        attended = E.engram_attention_step(layer.nr, seqs.cache, q, k, v, positions, seqs.slots(batch, positions), seqs.table,
                                           seqs.lens, workspace=workspace)
        logits = layer.logits(x, attended)
        for h, t in zip(history, token.tolist()):
            h.append(t)
        lookback = torch.cat([lookback[:, 1:], token_map[token.long()].unsqueeze(1)], 1).contiguous()
        token = logits.argmax(1).to(torch.int32)
    return logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=["bf16", "fp8"], default="bf16")
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args(argv)
    w = get_workload("tiny_bf16")
    layer = Layer(w, seed=3)
    rng = np.random.default_rng(3)
    history = [rng.integers(0, w.raw_vocab, size=n).tolist() for n in (5, 40, 17)]
    longest = max(len(h) for h in history) + a.steps
    seqs = Sequences(len(history), longest, a.cache)
    first = prompt(layer, seqs, [np.array(h) for h in history]).argmax(1).to(torch.int32)
    stepped = decode(layer, seqs, history, first, a.steps)
    # the same tokens as prompts
    again = prompt(layer, Sequences(len(history), longest, a.cache), [np.array(h) for h in history])
    off = float((stepped - again).abs().max() / again.abs().max())
    same = bool((stepped.argmax(1) == again.argmax(1)).all())
    for h in history:
        print(len(h), "tokens, the last ten:", h[-10:])
    print(f"{a.cache} cache: decoded against prompted logits differ by {off:.2e} of the largest, next tokens {'equal' if same else 'differ'}")
    return off, same


if __name__ == "__main__":
    main()
