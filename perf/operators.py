"""Cases of the serving operators that stand next to the compressed weights: products with low-rank adapters of many
requests, a paged key/value cache held in 8 bits, the attention that reads it, and the upkeep of its pages.

Each case runs in one of two ways.  With `own` false, `run` computes the operator in its plain form: elementary torch
operations in fp32.  With `own` true, it makes the calls that a user of the package makes.  Both work on the tensors that
`prepare` makes from the seed.

What the operators compute:

lora    Y[t] = W x_t + s_a B_a (A_a x_t), a = the adapter of token t (none: W x_t alone).  With `base` W is a matrix in
        the fixed-width form and Y is made in the call; without it Y is given and the adapters' part is added to it.
append  New tokens' keys and values go to their slots of the cache.  One scale (a power of two) per page, head and
        side: the least 2^e (e >= -60) with |x| <= Q 2^e for every value of the page (Q = 448 for e4m3, 127 for int8).
        Tokens that are in the page already are rounded again when it grows.
attend  softmax(q k / sqrt(dim)) v over the tokens a query sees: those up to its own place, of these the last
        `window` (0: all) and the first `sinks`; with `softcap` c the logits are c tanh(logit / c).  A query's place is
        counted from the end of its sequence.
fork    Children share the whole pages of a parent and get a copy of its last, partly filled page; then every child
        grows by some tokens, and at the end the children are freed.
compact Pages in use move to the lowest places of the pool, those above into the holes below, in order.

The cache: k [layers, pages, kv_heads, page, D] and v [layers, pages, kv_heads, D, page] bytes (D: dim rounded up to a
multiple of 64, zeros past dim), scale [layers, pages, kv_heads, 2] fp32, refs [pages], table [rows, pages per row] and
lens [rows] int32.  A free page is one with refs 0, and the lowest free page is taken first.
"""
import math
import random

import torch

own = False

LARGEST = {"e4m3": 448.0, "int8": 127.0}


def listed():
    return [
        # one request with an adapter, on a 4096 x 4096 projection: the latency of a lone user's token
        {"name": "lora one token", "op": "lora", "tokens": 1, "rows": 4096, "cols": 4096, "adapters": 8, "rank": 16,
         "mixed": False, "base": True, "y32": True},
        # a full decode batch, nearly every request with another adapter, on the layer's down projection
        {"name": "lora 64 requests", "op": "lora", "tokens": 64, "rows": 3584, "cols": 14336, "adapters": 64, "rank": 64,
         "mixed": True, "base": True, "y32": True},
        # prompts of several requests, beside a projection that the caller has done (gate/up of the layer)
        {"name": "lora prompts", "op": "lora", "tokens": 4097, "rows": 14336, "cols": 3584, "adapters": 5, "rank": 32,
         "mixed": True, "base": False, "y32": False},
        # one decode step's keys and values of 64 sequences (Gemma-2-9B-shaped heads)
        {"name": "append a step", "op": "append", "seqs": 64, "new": 1, "context": 2048, "kv_heads": 8, "dim": 256,
         "page": 64, "type": "int8", "ragged": 3},
        # four ragged prompts' keys and values (the 27.7B checkpoint's heads)
        {"name": "append prompts", "op": "append", "seqs": 4, "new": 8191, "context": 8191, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "e4m3", "ragged": 4},
        # a lone user's token over a short context
        {"name": "attend one short", "op": "attend", "seqs": 1, "new": 1, "context": 777, "heads": 16, "kv_heads": 8,
         "dim": 256, "page": 16, "type": "e4m3", "window": 0, "sinks": 0, "softcap": 50.0, "ragged": 0},
        # a ragged decode batch on a layer with a sliding window, the first tokens kept
        {"name": "attend window batch", "op": "attend", "seqs": 64, "new": 1, "context": 8192, "heads": 16,
         "kv_heads": 8, "dim": 256, "page": 64, "type": "e4m3", "window": 4096, "sinks": 4, "softcap": 50.0, "ragged": 5},
        # few sequences of long documents, five query heads to a key head
        {"name": "attend long", "op": "attend", "seqs": 4, "new": 1, "context": 131071, "heads": 40, "kv_heads": 8,
         "dim": 128, "page": 32, "type": "int8", "window": 0, "sinks": 0, "softcap": 0.0, "ragged": 0},
        # a chunk of two prompts over what the cache holds of them
        {"name": "attend prompts", "op": "attend", "seqs": 2, "new": 2048, "context": 8000, "heads": 40, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "e4m3", "window": 0, "sinks": 0, "softcap": 0.0, "ragged": 6},
        # one conversation branched once
        {"name": "fork one", "op": "fork", "layers": 2, "parents": 1, "children": 1, "context": 100, "new": 1,
         "kv_heads": 8, "dim": 128, "page": 16, "type": "e4m3", "ragged": 0},
        # several samples of each of a few prompts, through all layers of a model
        {"name": "fork samples", "op": "fork", "layers": 42, "parents": 4, "children": 8, "context": 3000, "new": 40,
         "kv_heads": 8, "dim": 256, "page": 16, "type": "int8", "ragged": 7},
        # a pool with holes, closed up through all layers
        {"name": "compact pool", "op": "compact", "layers": 42, "pages": 1021, "used": 0.6, "rows": 48, "kv_heads": 8,
         "dim": 256, "page": 16, "type": "e4m3", "ragged": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "append", "attend", "attend", "fork", "compact"])
    kind, ragged = rng.choice(["e4m3", "int8"]), rng.randint(1, 1 << 20)
    if op == "lora":
        base = rng.random() < 0.5
        # the fixed-width form's batched product takes columns in multiples of 2048 and batches of up to 64
        return {"op": "lora", "tokens": _log(rng, 1, 64) if base else _log(rng, 1, 4097), "rows": _log(rng, 64, 14336),
                "cols": 2048 * rng.randint(1, 7) if base else _log(rng, 64, 3584), "adapters": _log(rng, 1, 64),
                "rank": _log(rng, 1, 64), "mixed": rng.random() < 0.5, "base": base, "y32": base or rng.random() < 0.5}
    if op == "fork" or op == "compact":
        shape = {"layers": _log(rng, 1, 42), "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 96, 128, 256]),
                 "page": rng.choice([16, 32, 64]), "type": kind, "ragged": ragged}
        if op == "compact":
            while shape["layers"] * shape["kv_heads"] * shape["dim"] * shape["page"] > 42 * 8 * 256 * 16:
                shape["layers"] = max(1, shape["layers"] // 2)
            return {"op": op, "pages": _log(rng, 64, 1021), "used": rng.uniform(0.2, 0.9), "rows": _log(rng, 4, 48), **shape}
        context = _log(rng, 1, 3000)
        while shape["layers"] * shape["kv_heads"] * shape["dim"] * (context + 64) > 42 * 8 * 256 * 3000:
            context = max(1, context // 2)
        return {"op": op, "parents": _log(rng, 1, 4), "children": _log(rng, 1, 8), "context": context,
                "new": _log(rng, 1, 40), **shape}
    page, dim, kv_heads = rng.choice([16, 32, 64, 128]), rng.choice([64, 80, 96, 128, 256]), rng.choice([1, 2, 4, 8])
    wider = max(1, kv_heads * dim // 1024)
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, 32764 // (seqs * wider) + 2)
        return {"op": op, "seqs": seqs, "new": new, "context": new + _log(rng, 1, 2048), "kv_heads": kv_heads, "dim": dim,
                "page": page, "type": kind, "ragged": ragged}
    seqs = _log(rng, 1, 64)
    tokens = 524284 // (seqs * wider)
    new = 1 if rng.random() < 0.6 else _log(rng, 2, 2048 // seqs + 2)
    context = _log(rng, max(new, 16), min(tokens, 131071) if new == 1 else max(new, 8000))
    return {"op": op, "seqs": seqs, "new": new, "context": context, "heads": kv_heads * rng.choice([1, 2, 4, 5]),
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind,
            "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "sinks": rng.choice([0, 4]),
            "softcap": rng.choice([0.0, 50.0]), "ragged": ragged}


# ---------------------------------------------------------------- shapes that a case stands for
def _lengths(case, n, top):
    """n lengths up to `top`: all equal, or the longest first and the others spread over an eighth to the whole of it."""
    if not case["ragged"]:
        return [top] * n
    rng = random.Random(case["ragged"])
    return [top] + [min(top, _log(rng, max(1, top // 8), top)) for _ in range(n - 1)]


def _new_counts(case):
    if case["new"] == 1 or not case["ragged"]:
        return [case["new"]] * case["seqs"]
    rng = random.Random(case["ragged"] + 1)
    return [case["new"]] + [rng.randint(max(1, case["new"] // 2), case["new"]) for _ in range(case["seqs"] - 1)]


def _wide(dim):
    return -(-dim // 64) * 64


def _adapter_ranks(case):
    """The ranks of the adapters: all `rank`, or spread from a quarter of it to the whole."""
    if not case["mixed"]:
        return [case["rank"]] * case["adapters"]
    rng = random.Random(case["rank"] * 1000 + case["adapters"])
    return [rng.randint(max(1, case["rank"] // 4), case["rank"]) for _ in range(case["adapters"])]


def _adapter_of(case):
    """The adapter of each token (-1: none): one per request in a decode batch, runs of tokens for prompts."""
    rng = random.Random(case["tokens"] * 31 + case["adapters"])
    n, t = case["adapters"], case["tokens"]
    if t == 1:
        return [rng.randrange(n)]
    if t <= 64:
        first = list(range(n))
        rng.shuffle(first)
        return [-1 if i % 16 == 15 else first[i % n] for i in range(t)]
    got = []
    while len(got) < t:
        got += [rng.randint(-1, n - 1)] * rng.randint(1, max(1, t // 6))
    return got[:t]


def work(case):
    op = case["op"]
    if op == "lora":
        t, rows, cols = case["tokens"], case["rows"], case["cols"]
        ranks, of = _adapter_ranks(case), _adapter_of(case)
        adapters = sum(ranks[a] for a in set(of) if a >= 0) * 2 * (rows + cols)
        flops = sum(ranks[a] for a in of if a >= 0) * 2 * (rows + cols)
        y = t * rows * (4 if case["y32"] else 2)
        if case["base"]:      # the fixed-width form holds 11 bits a weight
            return {"bytes": rows * cols * 11 // 8 + adapters + 2 * t * cols + y, "flops": flops + 2 * t * rows * cols}
        with_one = sum(a >= 0 for a in of) / t
        return {"bytes": adapters + with_one * (2 * t * cols + 2 * y), "flops": flops}
    if op == "append":
        n = sum(_new_counts(case)) * case["kv_heads"] * case["dim"] * 2
        return {"bytes": n * 2 + n, "flops": 2 * n}
    if op == "attend":
        lens, new = _lengths(case, case["seqs"], case["context"]), _new_counts(case)
        pairs = seen = 0
        for length, q in zip(lens, new):
            q = min(q, length)
            w = case["window"] or length + 1
            s = case["sinks"] if case["window"] else 0
            for p in range(length - q, length):
                pairs += min(p + 1, w) + min(s, max(0, p + 1 - w))
            seen += min(length, w + q - 1) + min(s, max(0, length - w - q + 1))
        rows = sum(new) * case["heads"]
        return {"bytes": seen * case["kv_heads"] * case["dim"] * 2 + rows * case["dim"] * 4 + 4 * rows,
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    page = 2 * case["kv_heads"] * (case["page"] * case["dim"] + 4) * case["layers"]
    if op == "fork":
        lens = _lengths(case, case["parents"], case["context"])
        copies = sum(n % case["page"] > 0 for n in lens) * case["children"]
        held = sum(-(-(n + case["new"]) // case["page"]) for n in lens) * case["children"]
        return {"bytes": 2 * copies * page + 16 * held, "flops": 0}
    rng = random.Random(case["ragged"])
    used = [rng.random() < case["used"] for _ in range(case["pages"])]
    moved = sum(used[sum(used):])
    return {"bytes": 2 * moved * page + 16 * case["pages"], "flops": 0}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _heads_like(g, *shape):
    """Keys or values as projections give them: channels of differing size, now and then a large one."""
    dim = shape[-1]
    size = torch.exp(0.4 * torch.randn(dim, generator=g, device="cuda"))
    size[torch.rand(dim, generator=g, device="cuda") < 0.02] *= 6.0
    return torch.randn(*shape, generator=g, device="cuda") * size


def _values(codes, kind):
    """The values that 8-bit codes stand for, before their scale."""
    return codes.view(torch.float8_e4m3fn if kind == "e4m3" else torch.int8).float()


def _codes(x, kind):
    """Values within the type's range to the nearest code, ties to even."""
    if kind == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _scale_for(amax, kind):
    """The least power of two s >= 2^-60 with amax <= LARGEST s, exactly."""
    m, e = torch.frexp(amax / 2.0 ** (9 if kind == "e4m3" else 7))
    e = e + (m > (0.875 if kind == "e4m3" else 127.0 / 128.0)).int()
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp_min(-60)
    return ((e + 127) << 23).view(torch.float32)


def _pool(case, g, layers, pages, rows, per_row, lens, room=None):
    """A filled cache: rows of `lens` tokens on randomly placed pages, with pages for `room` tokens (default: lens); what
    no row holds is stale bytes."""
    page, h, dim, kind = case["page"], case["kv_heads"], case["dim"], case["type"]
    wide = _wide(dim)
    need = [-(-n // page) for n in room or lens]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((rows, per_row), -1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(pages, dtype=torch.int32, device="cuda")   # tokens that each page holds
    at = 0
    for i, n in enumerate(need):
        ids = order[at:at + n]
        at += n
        table[i, :n] = ids
        slots[ids.long()] = (lens[i] - page * torch.arange(n, device="cuda")).clamp(0, page).int()
    held = torch.arange(page, device="cuda")[None, :] < slots[:, None]
    k = torch.zeros(layers, pages, h, page, wide, dtype=torch.uint8, device="cuda")
    v = torch.zeros(layers, pages, h, wide, page, dtype=torch.uint8, device="cuda")
    scale = torch.empty(layers, pages, h, 2, device="cuda")
    for layer in range(layers):
        x = _heads_like(g, pages, h, page, dim)
        s = _scale_for((x * held[:, None, :, None]).abs().amax((2, 3)), kind)
        scale[layer, :, :, 0] = s
        stale = torch.randint(0, 256, (pages, h, page, dim), generator=g, device="cuda", dtype=torch.uint8)
        k[layer, ..., :dim] = torch.where(held[:, None, :, None], _codes(x / s[..., None, None], kind), stale)
        x = _heads_like(g, pages, h, page, dim).transpose(2, 3)
        s = _scale_for((x * held[:, None, None, :]).abs().amax((2, 3)), kind)
        scale[layer, :, :, 1] = s
        v[layer, ..., :dim, :] = torch.where(held[:, None, None, :], _codes(x / s[..., None, None], kind),
                                             stale.transpose(2, 3))
    all_lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    all_lens[:len(lens)] = _ints(room or lens)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:at].long()] = 1
    return {"k": k, "v": v, "scale": scale, "refs": refs, "table": table, "lens": all_lens}


def _cache(case, pool):
    """The package's cache over the pool's own tensors."""
    from lossless_entropy_coding_amd import kv
    return kv.KvCache.over(pool["k"], pool["v"], pool["scale"], pool["refs"], pool["table"], pool["lens"],
                           head_dim=case["dim"], dtype=case["type"])


def _starts(counts):
    return _ints([0] + list(torch.tensor(counts).cumsum(0).tolist()))


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "lora":
        t, rows, cols, n, r = (case[x] for x in ("tokens", "rows", "cols", "adapters", "rank"))
        ranks = _ints(_adapter_ranks(case))
        live = torch.arange(r, device="cuda")[None, :] < ranks[:, None]
        s = {"x": torch.randn(t, cols, generator=g, device="cuda").bfloat16(), "ranks": ranks.tolist(),
             "a": (torch.randn(n, r, cols, generator=g, device="cuda") * cols ** -0.5 * live[:, :, None]).bfloat16(),
             "b": (torch.randn(n, rows, r, generator=g, device="cuda") * 0.05 * live[:, None, :]).bfloat16(),
             "factor": 0.5 + torch.rand(n, generator=g, device="cuda"), "of": _ints(_adapter_of(case))}
        if case["base"]:
            s["w"] = (torch.randn(rows, cols, generator=g, device="cuda") * 0.02).bfloat16()
        else:
            y = torch.randn(t, rows, generator=g, device="cuda")
            s["y"] = y if case["y32"] else y.bfloat16()
        return s
    if op == "append":
        new, h, dim = _new_counts(case), case["kv_heads"], case["dim"]
        lens = [max(a, b) for a, b in zip(_lengths(case, case["seqs"], case["context"]), new)]
        need = sum(-(-n // case["page"]) for n in lens)
        # the rows' lengths count the new tokens already
        s = _pool(case, g, 1, need + need // 16 + 1, case["seqs"], -(-max(lens) // case["page"]),
                  [a - b for a, b in zip(lens, new)], lens)
        s["fresh_k"] = _heads_like(g, sum(new), h, dim).bfloat16()
        s["fresh_v"] = _heads_like(g, sum(new), h, dim).bfloat16()
        s["seqs"], s["starts"], s["most"] = _ints(list(range(case["seqs"]))), _starts(new), max(new)
        return s
    if op == "attend":
        lens, new = _lengths(case, case["seqs"], case["context"]), _new_counts(case)
        need = sum(-(-n // case["page"]) for n in lens)
        s = _pool(case, g, 1, need + need // 16 + 1, case["seqs"], -(-max(lens) // case["page"]), lens)
        s["q"] = (torch.randn(sum(new), case["heads"], case["dim"], generator=g, device="cuda")).bfloat16()
        s["seqs"], s["starts"], s["most"] = _ints(list(range(case["seqs"]))), _starts(new), max(new)
        s["longest"] = max(lens)
        return s
    if op == "fork":
        page, lens = case["page"], _lengths(case, case["parents"], case["context"])
        n = case["parents"] * case["children"]
        need = sum(-(-x // page) for x in lens)
        grown = sum(-(-(x + case["new"]) // page) - x // page for x in lens) * case["children"]
        s = _pool(case, g, case["layers"], need + grown + 7, case["parents"] + n, -(-(max(lens) + case["new"]) // page), lens)
        s["parents"] = _ints([i for i in range(case["parents"]) for _ in range(case["children"])])
        s["kids"] = _ints([case["parents"] + i for i in range(n)])
        s["grow"] = _ints([case["new"]] * n)
        return s
    rng = random.Random(case["ragged"])
    used = [i for i in range(case["pages"]) if rng.random() < case["used"]]
    cut = sorted(rng.randint(0, len(used)) for _ in range(case["rows"] - 1))
    held = [b - a for a, b in zip([0] + cut, cut + [len(used)])]
    lens = [max(0, n * case["page"] - rng.randrange(case["page"])) for n in held]
    s = _pool(case, g, case["layers"], case["pages"], case["rows"], max(held) + 1, [])
    mixed = torch.tensor(used, dtype=torch.int32, device="cuda")[torch.randperm(len(used), generator=g, device="cuda")]
    at = 0
    for i, n in enumerate(held):
        s["table"][i, :n] = mixed[at:at + n]
        at += n
    s["lens"].copy_(_ints(lens))
    s["refs"][mixed.long()] = 1
    s["new_table"], s["new_refs"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:       # what a serving program keeps between calls: compressed weights, laid-out adapters, the cache's handle
        if case["op"] == "lora":
            from lossless_entropy_coding_amd import codec, lora
            s["pack"] = lora.LoraPack([(s["a"][i, :r], s["b"][i, :, :r], f)
                                       for i, (r, f) in enumerate(zip(s["ranks"], s["factor"].tolist()))])
            s["batch"] = lora.LoraBatch(s["of"], case["adapters"])
            if case["base"]:
                s["weights"] = codec.FixedPlan(codec.fixed_encode_device(s["w"]))
        else:
            s["cache"] = _cache(case, s)
    return s


# ---------------------------------------------------------------- the plain forms
def _lora_plain(s, case):
    """Every adapter's inner product with every token, those of other adapters set to zero, then the outer products."""
    n, r, x = case["adapters"], case["rank"], s["x"].float()
    mine = (s["of"][:, None] == torch.arange(n, device="cuda")[None, :]) * s["factor"][None, :]
    inner = (x @ s["a"].float().reshape(n * r, -1).T).reshape(-1, n, r) * mine[:, :, None]
    y = inner.reshape(-1, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    if case["base"]:
        return y + x @ s["w"].float().T
    return (y + s["y"].float()).to(s["y"].dtype)


def _append_plain(s, case):
    page, kind, dim = case["page"], case["type"], case["dim"]
    total = s["fresh_k"].shape[0]
    t = torch.arange(total, dtype=torch.int32, device="cuda")
    row = torch.searchsorted(s["starts"][1:].contiguous(), t, right=True)
    place = s["lens"][row] - s["starts"][row + 1] + t      # the rows' lengths count the new tokens
    where, slot = s["table"][row, place // page].long(), place % page
    pages, which = torch.unique(where, return_inverse=True)
    first = torch.full((len(pages),), page, dtype=slot.dtype, device="cuda").scatter_reduce(0, which, slot, "amin")
    older = torch.arange(page, device="cuda")[None, :] < first[:, None]
    for_all = which[:, None].expand(-1, case["kv_heads"])
    _page_side(s["k"], s["scale"], 0, s["fresh_k"], pages, which, slot, first, older, for_all, kind, dim)
    _page_side(s["v"].transpose(3, 4), s["scale"], 1, s["fresh_v"], pages, which, slot, first, older, for_all, kind, dim)
    eight = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    return {"k": s["k"].view(eight), "v": s["v"].view(eight), "scale": s["scale"]}


def _page_side(codes, scale, side, fresh, pages, which, slot, first, older, for_all, kind, dim):
    """One side (keys or values, as [.., page, D]) of the touched pages: the scale, the older tokens and the new ones."""
    x = fresh.float()
    amax = torch.zeros(len(pages), x.shape[1], device="cuda").scatter_reduce(0, for_all, x.abs().amax(2), "amax")
    old = scale[0, pages, :, side] * (first > 0)[:, None]
    now = torch.maximum(old, _scale_for(amax, kind))
    before = codes[0, pages]
    again = _codes(_values(before.contiguous(), kind) * (old / now)[..., None, None], kind)
    codes[0, pages] = torch.where(older[:, None, :, None], again, before)
    codes[0, pages[which], :, slot, :dim] = _codes(x / now[which][..., None], kind)
    scale[0, pages, :, side] = now


def _attend_plain(s, case):
    page, kind, dim, h = case["page"], case["type"], case["dim"], case["kv_heads"]
    n, most, group = case["seqs"], s["most"], case["heads"] // h
    width = s["table"].shape[1]
    pages = s["table"].clamp_min(0).long()
    lens, count = s["lens"], s["starts"].diff()
    t = torch.arange(width * page, device="cuda")
    held = t[None, :] < lens[:, None]                                                    # [n, T]
    k = _values(s["k"][0, pages], kind) * s["scale"][0, pages, :, 0][..., None, None]     # [n, width, h, page, D]
    k = k[..., :dim].transpose(1, 2).reshape(n, h, width * page, dim)
    k = torch.where(held[:, None, :, None], k, torch.zeros((), device="cuda"))
    v = _values(s["v"][0, pages], kind) * s["scale"][0, pages, :, 1][..., None, None]
    v = v[..., :dim, :].permute(0, 2, 1, 4, 3).reshape(n, h, width * page, dim)
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device="cuda"))
    j = torch.arange(most, device="cuda")
    token = (s["starts"][:-1, None] + j[None, :]).clamp_max(s["q"].shape[0] - 1)          # [n, most]
    q = s["q"][token.long()].float().reshape(n, most, h, group, dim).permute(0, 2, 3, 1, 4).reshape(n, h, group * most, dim)
    logit = (q @ k.transpose(2, 3)) * dim ** -0.5
    if case["softcap"]:
        logit = case["softcap"] * torch.tanh(logit / case["softcap"])
    place = lens[:, None] - count[:, None] + j[None, :]                                   # [n, most]
    seen = (t[None, None, :] <= place[:, :, None]) & held[:, None, :]
    if case["window"]:
        seen &= (t[None, None, :] > place[:, :, None] - case["window"]) | (t < case["sinks"])[None, None, :]
    logit = logit.reshape(n, h, group, most, -1).masked_fill(~seen[:, None, None], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    out = (p / total.clamp_min(1e-38)).reshape(n, h, group * most, -1) @ v
    out = out.reshape(n, h, group, most, dim).permute(0, 3, 1, 2, 4).reshape(n, most, h * group, dim)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, most, h * group)
    real = j[None, :] < count[:, None]
    return {"out": out[real].bfloat16(), "lse": lse[real]}


def _take_free(refs, wanted):
    """The lowest free pages, one for each True of `wanted` in order (what the others get is of no use)."""
    free = torch.argsort((refs != 0).int(), stable=True)
    return free[(wanted.reshape(-1).cumsum(0) - 1).clamp_min(0)].reshape(wanted.shape)


def _fork_plain(s, case):
    page, table, refs, lens = case["page"], s["table"], s["refs"], s["lens"]
    src, dst = s["parents"].long(), s["kids"].long()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    whole, part = lens[src] // page, lens[src] % page > 0
    shared = col < whole[:, None]
    mine = _take_free(refs, part)
    last = table[src, whole.clamp_max(table.shape[1] - 1).long()].long()
    at, to = last[part], mine[part]
    s["k"][:, to], s["v"][:, to], s["scale"][:, to] = s["k"][:, at], s["v"][:, at], s["scale"][:, at]
    rows = torch.where(shared, table[src], table[dst])
    rows = torch.where((col == whole[:, None]) & part[:, None], mine[:, None].int(), rows)
    refs.scatter_add_(0, table[src].clamp_min(0).long().reshape(-1), shared.int().reshape(-1))
    refs[to] = 1
    # growth
    held = whole + part.int()
    grown = (lens[src] + s["grow"] + page - 1) // page
    fresh = (col >= held[:, None]) & (col < grown[:, None])
    ids = _take_free(refs, fresh)
    rows = torch.where(fresh, ids.int(), rows)
    refs[ids[fresh]] = 1
    table[dst] = rows
    # the end of the children
    gone = col < grown[:, None]
    refs.scatter_add_(0, rows.clamp_min(0).long().reshape(-1), -gone.int().reshape(-1))
    lens[dst] = 0
    return {name: s[name] for name in ("k", "v", "scale", "refs", "table", "lens")}


def _compact_plain(s, case):
    live = s["refs"] > 0
    place = torch.arange(len(live), device="cuda")
    below = place < live.sum()
    movers, holes = (live & ~below).nonzero()[:, 0], (~live & below).nonzero()[:, 0]
    s["k"][:, holes], s["v"][:, holes], s["scale"][:, holes] = s["k"][:, movers], s["v"][:, movers], s["scale"][:, movers]
    to = place.clone()
    to[movers] = holes
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    held = col * case["page"] < s["lens"][:, None]
    s["new_table"].copy_(torch.where(held, to[s["table"].clamp_min(0).long()].int(), -1))
    s["new_refs"].zero_()
    s["new_refs"][to[live]] = s["refs"][live]
    return {"k": s["k"], "v": s["v"], "scale": s["scale"], "table": s["new_table"], "refs": s["new_refs"]}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"lora": _lora_plain, "append": _append_plain, "attend": _attend_plain, "fork": _fork_plain,
                "compact": _compact_plain}[op](s, case)
    if op == "lora":
        if case["base"]:
            return s["weights"].gemm_lora(s["x"], case["rows"], case["cols"], s["pack"], s["batch"])
        return s["pack"].add(s["y"], s["x"], s["batch"], out=torch.empty_like(s["y"]))
    cache = s["cache"]
    if op == "append":
        cache.append(0, s["fresh_k"], s["fresh_v"], s["seqs"], s["starts"], max_new=s["most"])
        eight = torch.float8_e4m3fn if case["type"] == "e4m3" else torch.int8
        return {"k": s["k"].view(eight), "v": s["v"].view(eight), "scale": s["scale"]}
    if op == "attend":
        out, lse = cache.attend(0, s["q"], s["seqs"], s["starts"], max_new=s["most"], max_len=s["longest"],
                                window=case["window"], sinks=case["sinks"], softcap=case["softcap"], lse=True)
        return {"out": out, "lse": lse}
    if op == "fork":
        cache.fork(s["parents"], s["kids"])
        cache.extend(s["kids"], s["grow"])
        cache.free(s["kids"])
        return {name: s[name] for name in ("k", "v", "scale", "refs", "table", "lens")}
    cache.compact(table_out=s["new_table"], refs_out=s["new_refs"])
    return {"k": s["k"], "v": s["v"], "scale": s["scale"], "table": s["new_table"], "refs": s["new_refs"]}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    """What `run` returns, one adapter, token, or sequence and head at a time.  Copies and page numbers have no such value."""
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    s = _inputs(case, seed)
    if op == "lora":
        x = s["x"].double()
        y = x @ s["w"].double().T if case["base"] else s["y"].double()
        for a in sorted(set(s["of"].tolist()) - {-1}):
            at = (s["of"] == a).nonzero()[:, 0]
            y[at] += float(s["factor"][a]) * ((x[at] @ s["a"][a].double().T) @ s["b"][a].double().T)
        return y
    page, kind, dim = case["page"], case["type"], case["dim"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    starts = s["starts"].tolist()
    if op == "append":
        k, v = _values(s["k"], kind).double(), _values(s["v"], kind).double()
        scale = s["scale"].double()
        for i in range(case["seqs"]):
            count = starts[i + 1] - starts[i]
            begin = lens[i] - count
            for j in range(begin // page, (lens[i] - 1) // page + 1):
                lo, hi = max(begin, j * page), min(lens[i], (j + 1) * page)
                fk = s["fresh_k"][starts[i] + lo - begin:starts[i] + hi - begin].double()
                fv = s["fresh_v"][starts[i] + lo - begin:starts[i] + hi - begin].double()
                p, a, b = table[i][j], lo - j * page, hi - j * page
                for side, f in ((0, fk), (1, fv)):
                    need = torch.ceil(torch.log2(f.abs().amax((0, 2)) / LARGEST[kind])).clamp_min(-60.0)
                    need = torch.exp2(torch.where(f.abs().amax((0, 2)) > 0, need, -60.0))
                    had = scale[0, p, :, side].clone() if a else torch.zeros_like(need)
                    now = torch.maximum(need, had)
                    scale[0, p, :, side] = now
                    if side == 0:
                        k[0, p, :, :a] *= (had / now)[:, None, None]
                        k[0, p, :, a:b, :dim] = f.transpose(0, 1) / now[:, None, None]
                    else:
                        v[0, p, :, :, :a] *= (had / now)[:, None, None]
                        v[0, p, :, :dim, a:b] = f.permute(1, 2, 0) / now[:, None, None]
        if kind == "int8":        # whole numbers: compared as they are
            return {"k": None, "v": None, "scale": scale}
        return {"k": k, "v": v, "scale": scale}
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        n, a, b = lens[i], starts[i], starts[i + 1]
        ids = s["table"][i, :-(-n // page)].long()
        t = torch.arange(n, device="cuda")
        place = (n - (b - a) + torch.arange(b - a, device="cuda"))[:, None]
        hidden = t[None, :] > place
        if case["window"]:
            hidden |= (t[None, :] <= place - case["window"]) & (t[None, :] >= case["sinks"])
        for h in range(case["kv_heads"]):
            k = _values(s["k"][0, ids, h], kind).double() * s["scale"][0, ids, h, 0].double()[:, None, None]
            v = _values(s["v"][0, ids, h].transpose(1, 2).contiguous(), kind).double() * s["scale"][0, ids, h, 1].double()[:, None, None]
            k, v = k.reshape(-1, k.shape[-1])[:n, :dim], v.reshape(-1, v.shape[-1])[:n, :dim]
            for m in range(h * group, (h + 1) * group):
                logit = s["q"][a:b, m].double() @ k.T / math.sqrt(dim)
                if case["softcap"]:
                    logit = case["softcap"] * torch.tanh(logit / case["softcap"])
                logit[hidden] = -math.inf
                lse[a:b, m] = torch.logsumexp(logit, -1)
                out[a:b, m] = torch.exp(logit - lse[a:b, m, None]).nan_to_num(0.0) @ v
    return {"out": out, "lse": lse}
