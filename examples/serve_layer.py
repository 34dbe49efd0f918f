"""One attention layer served from compressed weights: adapters of several
users beside the shared projections, a paged 8-bit key/value cache, prompts,
a fork, decode steps and the pool's upkeep.

    python examples/serve_layer.py [--steps N]

The layer's q, k, v and o projections are in the fixed-width form and are
never decoded to memory; every product adds the low-rank adapter of each
token's user.  The same layer is computed from the original weights with
plain torch operations in fp32, and the two are compared at every step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_entropy_coding_amd import codec, kv, lora  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM = 2048, 16, 4, 128
SHAPES = {"q": (HEADS * DIM, HIDDEN), "k": (KV_HEADS * DIM, HIDDEN), "v": (KV_HEADS * DIM, HIDDEN), "o": (HIDDEN, HEADS * DIM)}
USERS = 3                      # adapters; users come without one, too


class ServedLayer:
    """The projections, their adapters and the cache."""

    def __init__(self, weights, adapters, rows, pages):
        self.plans = {n: codec.FixedPlan(codec.fixed_encode_device(w)) for n, w in weights.items()}
        self.packs = {n: lora.LoraPack(a) for n, a in adapters.items()}
        self.cache = kv.KvCache(layers=1, kv_heads=KV_HEADS, head_dim=DIM, n_pages=pages, max_seqs=rows, max_pages=pages,
                                page_tokens=16, dtype="int8")

    def project(self, name, x, batch):
        r, c = SHAPES[name]
        return self.plans[name].gemm_lora(x, r, c, self.packs[name], batch)

    def __call__(self, x, rows, counts, users):
        """x: (tokens, hidden) bfloat16, counts[i] tokens of cache row rows[i],
        in order; users: the adapter of each token.  Returns (tokens, hidden)
        fp32.  Up to 64 tokens a call, as the batched product takes."""
        t = x.shape[0]
        batch = lora.LoraBatch(users, USERS)
        ids = torch.tensor(rows, dtype=torch.int32, device="cuda")
        n = torch.tensor(counts, dtype=torch.int32, device="cuda")
        starts = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
        q = self.project("q", x, batch).bfloat16().view(t, HEADS, DIM)
        k = self.project("k", x, batch).view(t, KV_HEADS, DIM)              # fp32 straight into the cache
        v = self.project("v", x, batch).view(t, KV_HEADS, DIM)
        self.cache.extend(ids, n)
        self.cache.append(0, k, v, ids, starts, max_new=max(counts))
        out = self.cache.attend(0, q, ids, starts, max_new=max(counts), window=256, sinks=4)
        return self.project("o", out.view(t, HEADS * DIM), batch)


class PlainLayer:
    """The same from the original weights, with the keys and values of each row in fp32."""

    def __init__(self, weights, adapters, rows):
        self.weights, self.adapters = weights, adapters
        self.k, self.v = ([torch.zeros(0, KV_HEADS, DIM, device="cuda") for _ in range(rows)] for _ in range(2))

    def project(self, name, x, users):
        y = x.float() @ self.weights[name].float().T
        for i, (a, b, s) in enumerate(self.adapters[name]):
            mine = users == i
            y[mine] += s * (x[mine].float() @ a.float().T) @ b.float().T
        return y

    def __call__(self, x, rows, counts, users):
        t = x.shape[0]
        q = self.project("q", x, users).view(t, HEADS, DIM)
        k, v = self.project("k", x, users).view(t, KV_HEADS, DIM), self.project("v", x, users).view(t, KV_HEADS, DIM)
        out, at = torch.empty(t, HEADS, DIM, device="cuda"), 0
        for r, n in zip(rows, counts):
            self.k[r], self.v[r] = torch.cat([self.k[r], k[at:at + n]]), torch.cat([self.v[r], v[at:at + n]])
            length = self.k[r].shape[0]
            place, token = torch.arange(length - n, length, device="cuda")[:, None], torch.arange(length, device="cuda")[None, :]
            seen = (token <= place) & ((token > place - 256) | (token < 4))
            for h in range(HEADS):
                g = h // (HEADS // KV_HEADS)
                p = (q[at:at + n, h] @ self.k[r][:, g].T * DIM ** -0.5).masked_fill(~seen, -torch.inf).softmax(-1)
                out[at:at + n, h] = p @ self.v[r][:, g]
            at += n
        return self.project("o", out.view(t, HEADS * DIM).bfloat16(), users)

    def fork(self, parent, child):
        self.k[child], self.v[child] = self.k[parent].clone(), self.v[parent].clone()

    def free(self, r):
        self.k[r], self.v[r] = self.k[r][:0], self.v[r][:0]


def run(steps: int = 8, seed: int = 0, log=print) -> float:
    """Two prompts, a fork, decode steps, an ended row, a compaction, more
    steps; returns the largest relative distance (2-norm) from the plain layer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    weights = {n: (rand(*s) * s[1] ** -0.5).bfloat16() for n, s in SHAPES.items()}
    adapters = {n: [((rand(r, c) * c ** -0.5).bfloat16(), (rand(rows, r) * 0.1).bfloat16(), 1.0 + i)
                    for i, r in enumerate((8, 16, 5))] for n, (rows, c) in SHAPES.items()}
    served, plain = ServedLayer(weights, adapters, rows=6, pages=200), PlainLayer(weights, adapters, rows=6)
    worst = 0.0

    def step(rows, counts, users):
        nonlocal worst
        who = torch.tensor([u for u, n in zip(users, counts) for _ in range(n)], dtype=torch.int32, device="cuda")
        x = rand(sum(counts), HIDDEN).bfloat16()
        a, b = served(x, rows, counts, who), plain(x, rows, counts, who)
        off = float((a - b).norm() / b.norm())
        worst = max(worst, off)
        return off

    for _ in range(6):                                   # two prompts in chunks of up to 64 tokens
        off = step([0, 1], [40, 24], [0, -1])
    log(f"prompts of 240 and 144 tokens: {off:.4f} from the plain layer")
    served.cache.fork(torch.tensor([0, 0], dtype=torch.int32, device="cuda"), torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    plain.fork(0, 2), plain.fork(0, 3)
    rows, users = [0, 1, 2, 3], [0, -1, 1, 2]
    for _ in range(steps):
        off = step(rows, [1] * 4, users)
    log(f"{steps} decode steps of 4 rows, two of them forked: {off:.4f}")
    served.cache.free(torch.tensor([0], dtype=torch.int32, device="cuda"))
    plain.free(0)
    served.cache.compact()
    for _ in range(steps):
        off = step(rows[1:], [1] * 3, users[1:])
    served.cache.check()
    used = int((served.cache.refs > 0).sum())
    assert int(served.cache.refs[:used].min()) > 0, "pages in use are the lowest after a compaction"
    log(f"{steps} more after the first row ended and the pool was compacted ({used} pages in use): {off:.4f}")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    print("largest distance: %.4f" % run(ap.parse_args().steps))
