"""A beam search served from compressed weights: the prompts of two requests go
through the cache once, every request goes on in several beams that share its
prompt's pages, and each step chooses the beams that live on.

    python examples/beam_search.py [--steps N]

The model is one attention layer between an embedding and an output projection,
with random weights, all but the embedding in the fixed-width form.  A step
is: the plan of its tokens, keys and values into the cache, attention that
reads each prompt once for all of its beams, logits, the choice, and the move
of the cache's rows to their parents.  The same step is computed from the
original weights with plain torch operations in fp32, on the history that the
search has chosen, and the two are compared at every step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_entropy_coding_amd import beam, codec, kv  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, END = 2048, 16, 4, 128, 4001, 7
SHAPES = {"q": (HEADS * DIM, HIDDEN), "k": (KV_HEADS * DIM, HIDDEN), "v": (KV_HEADS * DIM, HIDDEN), "o": (HIDDEN, HEADS * DIM),
          "head": (VOCAB, HIDDEN)}


def _ids(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Served:
    """The layer from compressed weights, with rows for every beam."""

    def __init__(self, weights, rows):
        self.embedding = weights["embedding"]
        self.plans = {n: codec.FixedPlan(codec.fixed_encode_device(weights[n])) for n in SHAPES}
        self.cache = kv.KvCache(layers=1, kv_heads=KV_HEADS, head_dim=DIM, n_pages=400, max_seqs=rows, max_pages=64, page_tokens=16,
                                dtype="int8")

    def project(self, name, x):
        return self.plans[name].gemm(x, *SHAPES[name])

    def __call__(self, tokens, rows, counts, groups=None):
        """tokens: (n) of the rows, counts[i] of row rows[i]; logits (n, vocab) fp32."""
        n, most = len(tokens), max(counts)
        x = self.embedding[tokens]
        ids, many = _ids(rows), _ids(counts)
        self.cache.extend(ids, many)
        plan = kv.KvBatch(self.cache, ids, many, groups=None if groups is None else _ids(groups), total=n, max_new=most)
        q = self.project("q", x).bfloat16().view(n, HEADS, DIM)
        k, v = (self.project(s, x).view(n, KV_HEADS, DIM) for s in ("k", "v"))
        self.cache.append(0, k, v, ids, plan.starts, max_new=most)
        y = self.cache.attend_shared(0, q, plan)
        y = x.float() + self.project("o", y.view(n, HEADS * DIM))
        self.shared = plan.shared
        return self.project("head", y.bfloat16())


class Plain:
    """The same from the original weights, with the keys and values of each row in fp32."""

    def __init__(self, weights, rows):
        self.weights = {n: w.float() for n, w in weights.items()}
        self.k, self.v = ([torch.zeros(0, KV_HEADS, DIM, device="cuda") for _ in range(rows)] for _ in range(2))

    def __call__(self, tokens, rows, counts):
        x = self.weights["embedding"][tokens]
        q, k, v = ((x @ self.weights[s].T).view(len(tokens), -1, DIM) for s in "qkv")
        out, at = torch.empty_like(q), 0
        for r, n in zip(rows, counts):
            self.k[r], self.v[r] = torch.cat([self.k[r], k[at:at + n]]), torch.cat([self.v[r], v[at:at + n]])
            length = self.k[r].shape[0]
            seen = torch.arange(length, device="cuda")[None, :] <= torch.arange(length - n, length, device="cuda")[:, None]
            for h in range(HEADS):
                g = h // (HEADS // KV_HEADS)
                p = (q[at:at + n, h] @ self.k[r][:, g].T * DIM ** -0.5).masked_fill(~seen, -torch.inf).softmax(-1)
                out[at:at + n, h] = p @ self.v[r][:, g]
            at += n
        return (x + out.reshape(len(tokens), HEADS * DIM) @ self.weights["o"].T) @ self.weights["head"].T

    def move(self, rows, parents):
        k, v = [self.k[r] for r in rows], [self.v[r] for r in rows]
        for r, p in zip(rows, parents):
            self.k[r], self.v[r] = k[p], v[p]


def run(steps: int = 10, requests: int = 2, beams: int = 4, prompt: int = 150, seed: int = 0, log=print):
    """The best answers' tokens, and the largest relative distance (2-norm) of a
    step's logits from the plain layer's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights = {n: (torch.randn(*s, generator=g, device="cuda") * s[1] ** -0.5).bfloat16() for n, s in SHAPES.items()}
    weights["head"] = (weights["head"].float() * 3).bfloat16()
    weights["embedding"] = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").bfloat16()
    rows = list(range(requests * beams))
    served, plain = Served(weights, len(rows)), Plain(weights, len(rows))
    chooser, worst = beam.Beams(requests, beams, eos=END), 0.0

    # the prompts, in chunks of 64 tokens in all (as the batched product takes), into the first row of each request
    chunk = 64 // requests
    lead = rows[::beams]
    tokens = torch.randint(0, VOCAB, (requests, prompt), generator=g, device="cuda")
    for a in range(0, prompt, chunk):
        part = tokens[:, a:a + chunk]
        logits = served(part.reshape(-1), lead, [part.shape[1]] * requests, groups=list(range(requests + 1)))
        plain(part.reshape(-1), lead, [part.shape[1]] * requests)
    for i in range(1, beams):
        served.cache.fork(_ids(lead), _ids([r + i for r in lead]))
    plain.move(rows, [r // beams * beams for r in rows])

    # the first choice goes on from one beam of each request
    logits = logits.view(requests, -1, VOCAB)[:, -1].repeat_interleave(beams, 0).contiguous()
    scores = torch.full((requests, beams), -torch.inf, device="cuda")
    scores[:, 0] = 0
    done, words = torch.zeros(len(rows), dtype=torch.int32, device="cuda"), [[] for _ in rows]
    groups, ids = list(range(0, len(rows) + 1, beams)), _ids(rows)
    for step in range(steps):
        best = chooser.select(logits, scores, done=done)
        parents = best.parents.view(-1)
        served.cache.reorder(ids, parents)
        plain.move(rows, parents.tolist())
        scores, done, chosen = best.scores, best.done.view(-1), best.tokens.view(-1)
        words = [words[p] + [t] for p, t in zip(parents.tolist(), chosen.tolist())]
        logits = served(chosen.long(), rows, [1] * len(rows), groups)
        want = plain(chosen.long(), rows, [1] * len(rows))
        worst = max(worst, float((logits - want).norm() / want.norm()))
    served.cache.check()
    log(f"{steps} steps of {requests} requests with {beams} beams, {int(served.shared.min())} tokens of each in common: "
        f"logits {worst:.4f} from the plain layer")
    for b in range(requests):
        log(f"request {b}: {scores[b, 0]:.3f} {words[b * beams]}")
    return words, worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=10)
    run(ap.parse_args().steps)
