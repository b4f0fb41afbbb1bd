"""An attention block served in 8 bits: int8 projections, norm and rotation of
queries and keys, a paged 8-bit key/value cache, and its page bookkeeping, as a
generation loop uses them.

    python examples/int8_decoder_block.py [--steps N]

Three prompts are written and answered token by token; then the first sequence
is forked (two continuations of one prompt share its full pages), one sequence
ends, and the pool is packed. At last a tree of drafted tokens is verified in one
step, with the log probabilities of a head's tokens. Each step is checked against the same block
computed densely in fp32 from the unquantized weights: the block's outputs stay
within the error that 8-bit weights, activations and cache make.

Weights are random; the shapes are those of one layer with 16 query heads, 4
key/value heads and head size 128.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from group_wise_affine_amd import qmm  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE, VOCABULARY = 2048, 16, 4, 128, 32, 4000


class Block:
    """qkv projection -> norm and rotation -> cache -> attention -> output projection."""

    def __init__(self, gen):
        def weight(n, k):
            w = (torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16).cuda()
            return w, *qmm.i8_quantize(w)   # one scale per output channel, once
        self.w_qkv, self.qkv, self.qkv_scale = weight((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.w_out, self.out, self.out_scale = weight(HIDDEN, Q_HEADS * DIM)
        _, self.head, self.head_scale = weight(VOCABULARY, HIDDEN)
        self.q_norm, self.k_norm = ((1 + 0.2 * torch.randn(DIM, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, DIM, 2) / DIM)).cuda()

    def __call__(self, x, positions, cache, table, lens, cu, parent=None):
        """x [T, HIDDEN]: the new tokens of every sequence, packed; with parent they
        are trees of drafts."""
        t = qmm.i8_linear(x, self.qkv, self.qkv_scale).view(len(x), Q_HEADS + 2 * KV_HEADS, DIM)
        q, k, v = t[:, :Q_HEADS], t[:, Q_HEADS:Q_HEADS + KV_HEADS], t[:, Q_HEADS + KV_HEADS:]
        qmm.qk_norm_rope(q, k, positions, self.inv_freq, self.q_norm, self.k_norm, out=(q, k))
        qmm.kv8_append(cache, k, v, table, lens, cu)
        if parent is None:
            a = qmm.kv8_attention(cache, q, table, lens, cu)
        else:
            a = qmm.kv8_attention_tree(cache, q, table, lens, cu, parent)
        return qmm.i8_linear(a.view(len(x), Q_HEADS * DIM), self.out, self.out_scale)

    def scores(self, y, tokens):
        """Log probabilities of the next tokens, and the three most likely ones."""
        return qmm.logprobs(qmm.i8_linear(y, self.head, self.head_scale), tokens, top=3)

    def dense(self, x):
        """The same for one whole sequence, fp32, causal."""
        t = (x.float() @ self.w_qkv.float().t()).view(len(x), Q_HEADS + 2 * KV_HEADS, DIM).transpose(0, 1)
        q, k, v = t[:Q_HEADS], t[Q_HEADS:Q_HEADS + KV_HEADS], t[Q_HEADS + KV_HEADS:]
        angle = torch.arange(len(x), device=x.device)[:, None] * self.inv_freq
        cos, sin = angle.cos(), angle.sin()

        def turned(y, weight):
            y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + 1e-6) * weight.float()
            a, b = y.chunk(2, 2)
            return torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        q, k = turned(q, self.q_norm), turned(k, self.k_norm)
        k, v = (y.repeat_interleave(Q_HEADS // KV_HEADS, 0).contiguous() for y in (k, v))
        s = (q.contiguous() @ k.transpose(1, 2).contiguous()) * DIM ** -0.5
        s = s.masked_fill(torch.ones(len(x), len(x), device=x.device).triu(1).bool(), -torch.inf)
        a = (s.softmax(-1) @ v).transpose(0, 1).reshape(len(x), Q_HEADS * DIM)
        return a @ self.w_out.float().t()


class Pool:
    """The cache's pages and the slots that hold sequences, all on the device."""

    def __init__(self, pages, slots, most_tokens):
        self.cache = qmm.Kv8Cache(pages, KV_HEADS, PAGE, DIM)
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((slots, -(-most_tokens // PAGE)), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(slots, dtype=torch.int32, device="cuda")

    def step(self, parent, lens):
        """Slot s continues slot parent[s] (-1: nothing) and gets room for lens[s] tokens."""
        as_ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        new = as_ints(lens)
        self.ref, self.table, short = qmm.kv8_update(self.cache, self.ref, self.table, self.lens,
                                                     as_ints(parent), new)
        assert short.item() == 0, "the pool is too small"
        self.lens = new

    def pack(self):
        self.ref, self.table, _, used = qmm.kv8_compact(self.cache, self.ref, self.table)
        return used.item()


def run(steps=40, seed=0):
    """Worst relative error of a step's outputs, and the pages in use at the end."""
    gen = torch.Generator().manual_seed(seed)
    token = lambda n: torch.randn(n, HIDDEN, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    block, pool = Block(gen), Pool(pages=64, slots=4, most_tokens=512)
    seqs = [token(77), token(130), token(1), token(0)]   # what each slot has read
    worst = 0.0

    def batch(new):
        """Where each sequence's new tokens start, and their positions."""
        pos = [i for x, n in zip(seqs, new) for i in range(len(x) - len(n), len(x))]
        return (torch.tensor([0] + [len(x) for x in new], device="cuda").cumsum(0).int(),
                torch.tensor(pos, device="cuda", dtype=torch.int32))

    def forward(new):
        nonlocal worst
        cu, pos = batch(new)
        y = block(torch.cat(new), pos, pool.cache, pool.table, pool.lens, cu)
        at = 0
        for x, n in zip(seqs, new):
            if len(n):
                want = block.dense(x)[-len(n):]
                err = (y[at:at + len(n)].float() - want).norm() / want.norm()
                worst = max(worst, err.item())
                at += len(n)

    def decode(parent):
        nonlocal seqs
        seqs = [torch.cat([seqs[p], token(1)]) if p >= 0 else token(0) for p in parent]
        pool.step(parent, [len(x) for x in seqs])
        forward([x[-1:] for x in seqs])

    pool.step([-1] * 4, [len(x) for x in seqs])
    forward(seqs)
    for _ in range(steps):
        decode([0, 1, 2, -1])
    decode([0, 1, 2, 0])        # the last slot continues the first sequence
    decode([0, -1, 2, 3])       # the second sequence has ended
    for _ in range(steps):
        decode([0, -1, 2, 3])
    used = pool.pack()
    decode([0, -1, 2, 3])

    # drafts behind the first sequence: two ways to go on, one of them for three tokens
    tree, drafts = [-1, 0, 1, 0, 3], token(5)
    before = seqs[0]
    seqs = [torch.cat([before, drafts])] + seqs[1:]
    pool.step([0, -1, 2, 3], [len(x) for x in seqs])
    cu, pos = batch([drafts, token(0), token(0), token(0)])
    paths = []
    for i, p in enumerate(tree):
        paths.append((paths[p] if p >= 0 else []) + [i])
        pos[i] = len(before) + len(paths[i]) - 1   # its depth, not its place
    parent = torch.tensor(tree, dtype=torch.int32, device="cuda")
    y = block(drafts, pos, pool.cache, pool.table, pool.lens, cu, parent)
    for i, path in enumerate(paths):
        want = block.dense(torch.cat([before, drafts[path]]))[-1]
        worst = max(worst, ((y[i].float() - want).norm() / want.norm()).item())
    logprob, entropy, ids, top = block.scores(y, torch.arange(5, dtype=torch.int32, device="cuda"))
    assert bool((logprob < 0).all() and (entropy > 0).all() and (top[:, 0] >= logprob).all())
    return worst, used


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    worst, used = run(ap.parse_args().steps)
    print(f"relative error against the dense fp32 block: at most {worst:.4f}; pages in use: {used} of 64")
