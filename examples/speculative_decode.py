"""Speculative decoding of a small pruned decoder with the library's operators.

    python examples/speculative_decode.py [--steps 24] [--cache e4m3] [--layers 4]

A decoder with random 2:4 weights: per layer the sparse products nm_spmm24
(QKV, output, gate+up, down) for the drafted nodes of a step as one batch,
nm_rope_append and nm_tree_attention between them, and after the last layer
nm_tree_verify.  The accepted path is committed by appending its rows again at
their final slots.  In place of a draft model there is a stand-in that has seen
the text: it proposes the tokens of a plain decoding, three quarters of them
right, with wrong siblings.  With temperature 0 the tokens are those of decoding
one token at a time, which ``--check`` compares.
"""
from __future__ import annotations

import argparse
import os
import random
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import sparse_spmv_memory_gb300 as nm

HIDDEN, FFN, Q_HEADS, KV_HEADS, DIM, VOCAB, PAGE = 1024, 2048, 8, 2, 128, 2048, 16
DTYPES = {"fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class Matrix:
    """A 2:4 pruned matrix and the workspace of its products."""

    def __init__(self, rows, cols, gen):
        w = torch.randn((rows, cols), generator=gen, device="cuda") * (cols ** -0.5) * 1.4
        self.values, self.masks = nm.nm_pack(w.half(), 2, 4)
        self.work = torch.zeros(nm.nm_spmm24_workspace_bytes(rows, cols, 8), dtype=torch.uint8,
                                device="cuda")

    def __call__(self, x):  # at most 8 tokens
        return nm.nm_spmm24(self.values, self.masks, x, workspace=self.work)


class Decoder:
    """Weights, the paged cache of one sequence, and a step over a tree of nodes."""

    def __init__(self, layers, cache, positions, seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        heads = Q_HEADS + 2 * KV_HEADS
        self.layers = [dict(qkv=Matrix(heads * DIM, HIDDEN, gen), o=Matrix(HIDDEN, Q_HEADS * DIM, gen),
                            up=Matrix(2 * FFN, HIDDEN, gen), down=Matrix(HIDDEN, FFN, gen))
                       for _ in range(layers)]
        self.embed, self.head = (torch.randn((VOCAB, HIDDEN), generator=gen, device="cuda").half()
                                 for _ in range(2))
        self.freq = nm.nm_rope_inv_freq(DIM, 500000.0, "banded", 8.0, 1.0, 4.0, 8192.0)
        pages = -(-positions // PAGE)
        # a layer's pages in an order of their own, as an allocator hands them out
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
        shape = (layers, pages, KV_HEADS, PAGE, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=DTYPES[cache], device="cuda") for _ in range(2))
        self.ks = self.vs = [None] * layers
        if cache != "fp16":
            self.ks, self.vs = (torch.zeros(shape[:-1], device="cuda") for _ in range(2))
        self.len = 0
        self.work = torch.zeros(nm.nm_tree_attention_workspace_bytes(1, Q_HEADS, KV_HEADS, DIM, 8),
                                dtype=torch.uint8, device="cuda")

    def slots(self, positions):
        p = positions.long()
        return self.table[0, p // PAGE].long() * PAGE + p % PAGE

    def step(self, tokens, parents):
        """Logits after every node of a tree (node 0: the last committed token), and
        the QKV outputs that ``commit`` needs."""
        n = len(tokens)
        depth, mask = [0] * n, [0] * n
        for i, p in enumerate(parents):
            depth[i] = depth[p] + 1 if i else 0
            mask[i] = (mask[p] if i else 0) | 1 << i
        place = torch.arange(n, device="cuda") + self.len          # where a node's row lies
        pos = (torch.tensor(depth, device="cuda") + self.len).to(torch.int32)
        mask = torch.tensor(mask, dtype=torch.int64, device="cuda")
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ctx = torch.tensor([self.len], dtype=torch.int32, device="cuda")
        x = self.embed[torch.tensor(tokens, device="cuda")]
        qkvs, slots = [], self.slots(place)
        for i, w in enumerate(self.layers):
            qkv = w["qkv"](norm(x))
            q = nm.nm_rope_append(qkv, self.k[i], self.v[i], pos, slots, self.freq, Q_HEADS,
                                  k_scale=self.ks[i], v_scale=self.vs[i])
            a, _ = nm.nm_tree_attention(q, self.k[i], self.v[i], self.table, ctx, start, n,
                                        tree_mask=mask, k_scale=self.ks[i], v_scale=self.vs[i],
                                        workspace=self.work if n <= 8 else None)
            x = x + w["o"](a.view(n, -1))
            gate, up = w["up"](norm(x)).float().chunk(2, -1)
            x = x + w["down"]((torch.nn.functional.silu(gate) * up).half())
            qkvs.append(qkv)
        return (norm(x).float() @ self.head.float().T) * 2 * HIDDEN ** -0.5, qkvs, pos

    def commit(self, path, qkvs, pos):
        """Append the accepted nodes' rows again where they stay: node path[i] at the
        context's end + i (its position already is that)."""
        rows = torch.tensor(path, device="cuda")
        slots = self.slots(torch.arange(len(path), device="cuda") + self.len)
        for i, qkv in enumerate(qkvs):
            nm.nm_rope_append(qkv[rows], self.k[i], self.v[i], pos[rows], slots, self.freq, Q_HEADS,
                              k_scale=self.ks[i], v_scale=self.vs[i], want_q=False)
        self.len += len(path)


def propose(text, rnd):
    """A tree of 7 drafted tokens and their parents: two chains from node 0, each
    token right three times out of four (a draft model goes here)."""
    def guess(i):
        right = i < len(text) and rnd.random() < 0.75
        return text[i] if right else rnd.randrange(VOCAB)
    return [guess(0), guess(0), guess(1), guess(1), guess(2), guess(2), guess(3)], [0, 0, 1, 2, 3, 4, 5]


def decode(layers, cache, steps, temperature, seed, text=None):
    """``steps`` tokens, and how many drafted ones were accepted; ``text``: what the
    draft knows (None: one token at a time)."""
    gen, rnd = torch.Generator("cuda").manual_seed(seed + 1), random.Random(seed)
    model = Decoder(layers, cache, 16 + 8 * (steps + 2), seed)
    out, last, accepted = [], 1, 0
    while len(out) < steps:
        tokens, parents = [last], [-1]
        if text is not None:
            more, par = propose(text[len(out):], rnd)
            tokens, parents = tokens + more, parents + par
        n = len(tokens)
        logits, qkvs, pos = model.step(tokens, parents)
        ints = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (tokens, parents, [0, n])]
        path, count, token = nm.nm_tree_verify(
            logits, *ints, n, accept=torch.rand(n, generator=gen, device="cuda"),
            race=torch.empty((1, VOCAB), device="cuda").exponential_(generator=gen).clamp_min_(1e-30),
            temperature=temperature)
        kept = path[0, :int(count[0])].tolist()
        model.commit(kept, qkvs, pos)
        accepted += len(kept) - 1
        last = int(token[0])
        out += [tokens[i] for i in kept[1:]] + [last]
    return out[:steps], accepted


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=24, help="tokens to decode")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--cache", choices=sorted(DTYPES), default="fp16")
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--check", action="store_true", help="compare with one token at a time")
    a = ap.parse_args(argv)
    plain, _ = decode(a.layers, a.cache, a.steps, 0.0, a.seed)
    out, accepted = decode(a.layers, a.cache, a.steps, a.temperature, a.seed, plain)
    print("tokens:", *out)
    print(f"{accepted} of the {a.steps} tokens were drafted")
    if a.check:
        print("one at a time:", "the same" if plain == out else plain)
        return 0 if plain == out else 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
