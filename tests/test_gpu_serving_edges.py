"""The serving operators on the GPU where they are used in less usual ways:
calls first made in a capture, cache entries that exist nowhere, values that
are not finite, soft caps of any size, long rows of every head size."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf16(rng, *shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).bfloat16()


def _f64(t):
    return t.cpu().float().numpy().astype(np.float64)


def _filled(rng, lens, size=1.0, **kw):
    """A cache and its model, with rows of these lengths in layer 0."""
    kw = dict(dict(layers=1, max_seqs=len(lens), page_tokens=64, dtype="e4m3"), **kw)
    page = kw["page_tokens"]
    need = [-(-n // page) for n in lens]
    kw = dict(dict(n_pages=sum(need) + 2, max_pages=max(need) + 1), **kw)
    cache, model = kv.KvCache(**kw), S.Cache(**kw)
    rows, at = list(range(len(lens))), [0] + [int(x) for x in np.cumsum(lens)]
    k, v = (_bf16(rng, at[-1], kw["kv_heads"], kw["head_dim"], size=size) for _ in range(2))
    cache.extend(_ids(*rows), _ids(*lens))
    model.extend(rows, lens)
    cache.append(0, k.cuda(), v.cuda(), _ids(*rows), _ids(*at), max_new=max(lens))
    model.append(0, _f64(k), _f64(v), rows, at)
    torch.cuda.synchronize()
    return cache, model


def test_attention_first_called_in_a_capture():
    """Graphs captured with no workspace made before: an eager call and a later
    graph that come before the first one's replay are right, and so is every
    replay."""
    rng = np.random.default_rng(41)
    cache, _ = _filled(rng, [3000, 2000, 100, 7], kv_heads=1, head_dim=64)
    q, rows = _bf16(rng, 4, 16, 64).cuda(), _ids(0, 1, 2, 3)
    fresh = lambda: kv.KvCache.over(cache.k, cache.v, cache.scale, cache.refs, cache.table, cache.lens, 64)   # noqa: E731
    want = {n: cache.attend(0, q[:n], rows[:n], lse=True) for n in (1, 2, 4)}
    twin = fresh()
    full = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    del full                                         # memory that is not zero, for whoever asks next
    for n in (1, 2):
        out, lse = torch.zeros(n, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(2):
                twin.attend(0, q[:n], rows[:n], out=out, lse=lse)
        graphs.append(g), outs.append((out, lse))
    got = twin.attend(0, q, rows, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[4][0]) and torch.equal(got[1], want[4][1])
    for _ in range(3):
        for i in (1, 0):
            outs[i][0].zero_(), outs[i][1].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], want[i + 1][0]) and torch.equal(outs[i][1], want[i + 1][1])
        got = twin.attend(0, q, rows)
        torch.cuda.synchronize()
        assert torch.equal(got, want[4][0])


def test_growth_by_more_pages_than_32_bits_count():
    """1024 rows of 2^22 pages each: the pages wanted are 2^32, a sum that wraps
    to 0 would let the rows grow with no pages of their own."""
    n, pages = 1024, 1 << 22
    cache = kv.KvCache(1, 1, 1, 64, n, pages, page_tokens=16)
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    for last in (16 * pages, 16 * pages - 15, 1, 0):
        counts = torch.full((n,), 16 * pages, dtype=torch.int32, device="cuda")
        counts[-1] = last
        cache.extend(rows, counts)
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 1, last
        cache.status.zero_()
        assert not cache.lens.any() and not cache.refs.any()
    cache.extend(rows[:64], torch.ones(64, dtype=torch.int32, device="cuda"))
    cache.check()
    assert torch.equal(cache.table[:64, 0], rows[:64]) and bool((cache.refs == 1).all())


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dim,dtype", [(64, "e4m3"), (80, "int8"), (256, "e4m3")])
def test_queries_that_are_not_finite(dim, dtype, new):
    """A query with a NaN gives NaN, its logarithm too, where it sees a token,
    and so does one with an infinity (infinity less infinity in the softmax)
    unless a cap makes its logits finite; 0 and -infinity where it sees none.
    The queries beside it, in its tile and its sequence, are right.  Split and
    unsplit."""
    print("not finite", dim, dtype, new, flush=True)
    rng = np.random.default_rng(dim + new)
    lens, heads = [5000, 3, 200], 4
    cache, model = _filled(rng, lens, kv_heads=2, head_dim=dim, dtype=dtype)
    starts = [0, new, 2 * new, 3 * new]
    at = _ids(*starts)
    q = _bf16(rng, 3 * new, heads, dim).cuda()
    odd = q.clone()
    bad = {(0, 1): "nan", (new - 1, 2): "inf", (2 * new, 0): "-inf", (3 * new - 1, 3): "nan"}
    if new > 3:
        bad[(new, 0)] = "nan"                        # before the row's first token
    for (t, h), x in bad.items():
        odd[t, h, dim - 1] = float(x)
    for kw in ({}, dict(window=300, sinks=2), dict(softcap=10.0), dict(scale=-0.5)):
        got, lse = cache.attend(0, odd, _ids(0, 1, 2), at, max_new=new, lse=True, **kw)
        cache.check()
        hit = torch.zeros(3 * new, heads, dtype=torch.bool, device="cuda")
        nans = hit.clone()
        for (t, h), x in bad.items():
            hit[t, h] = True
            nans[t, h] = x == "nan" or "softcap" not in kw
        out, ref, slack, spread = model.attend(0, _f64(q), [0, 1, 2], starts, **kw)
        blind = torch.from_numpy(np.isneginf(ref)).cuda()
        assert bool(blind[new, 0]) == (new > 3) and torch.equal(torch.isneginf(lse), blind) and not got[blind].any()
        assert torch.isnan(got[nans & ~blind]).all() and torch.isnan(lse[nans & ~blind]).all()
        rest = (~hit & ~blind).cpu().numpy()
        assert np.all((np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))[rest])
        assert np.all((np.abs(_f64(lse) - np.where(rest, ref, 0)) <= slack + 2.0 ** -20 * (1 + np.abs(ref)))[rest])


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dim,page,dtype", [(64, 64, "int8"), (128, 16, "e4m3"), (256, 32, "int8")])
def test_tokens_without_a_page_are_left_out(dim, page, dtype, new):
    """Few and many rows: entries past the pool, in the middle, at the first and the last page, and a whole row of them."""
    print("no page", dim, page, dtype, new, flush=True)
    rng = np.random.default_rng(dim + new)
    lens, heads = [700, 90, 150], 4
    cache, model = _filled(rng, lens, kv_heads=2, head_dim=dim, page_tokens=page, dtype=dtype)
    last = (lens[0] - 1) // page
    gone = {(0, 0): -1, (0, 2): 1 << 30, (0, 3): cache.n_pages, (0, last): -(1 << 31)}
    gone.update({(1, c): -7 for c in range(-(-lens[1] // page))})
    for (r, c), e in gone.items():
        cache.table[r, c] = e
    at = [0, new, 2 * new, 3 * new]
    q = _bf16(rng, 3 * new, heads, dim)
    for kw in ({}, dict(window=200, sinks=page), dict(softcap=20.0)):
        got, lse = cache.attend(0, q.cuda(), _ids(0, 1, 2), _ids(*at), max_new=new, lse=True, **kw)
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 4
        cache.status.zero_()
        out, ref, slack, spread = model.attend(0, _f64(q), [0, 1, 2], at, gone=list(gone), **kw)
        g, l = _f64(got), _f64(lse)
        empty = np.isneginf(ref)
        assert empty[new:2 * new].all() and np.array_equal(empty, np.isneginf(l)) and np.all(g[empty] == 0)
        assert np.all(np.abs(g - out) <= S.attend_bound(out, slack, spread)), float(np.abs(g - out).max())
        assert np.all(np.abs(l[~empty] - ref[~empty]) <= slack[~empty] + 2.0 ** -20 * (1 + np.abs(ref[~empty])))


@pytest.mark.parametrize("new,dim,dtype", [(1, 64, "int8"), (70, 128, "e4m3"), (9, 256, "e4m3"), (80, 80, "int8")])
def test_soft_caps_of_any_size(new, dim, dtype):
    """Logits of up to hundreds under caps from far below to far above them: the
    error is a share of the capped logit (of the cap up to 256), so that a cap
    far above the logits leaves them as they are."""
    print("caps", new, dim, dtype, flush=True)
    rng = np.random.default_rng(dim + new)
    lens = [400, 90]
    cache, model = _filled(rng, lens, kv_heads=1, head_dim=dim, dtype=dtype)
    q = _bf16(rng, 2 * new, 2, dim, size=20.0)
    at = [0, new, 2 * new]
    for cap in (1e-42, 1e-35, 1e-3, 30.0, 256.0, 257.0, 1e3, 1e4, 1e6, 1e20, 3e38, float("inf")):
        for scale in (0.0, -0.3, 1e-3):
            got, lse = cache.attend(0, q.cuda(), _ids(0, 1), _ids(*at), max_new=new, softcap=cap, scale=scale, lse=True)
            cache.check()
            out, ref, slack, spread = model.attend(0, _f64(q), [0, 1], at, scale=scale,
                                                   softcap=0.0 if cap == float("inf") else float(np.float32(cap)))
            assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread)), (cap, scale)
            assert np.all(np.abs(_f64(lse) - ref) <= slack + 2.0 ** -20 * (1 + np.abs(ref))), (cap, scale)


@pytest.mark.parametrize("new", [1, 70])
def test_windows_and_sinks_past_every_row(new):
    rng = np.random.default_rng(new)
    cache, _ = _filled(rng, [500, 80], kv_heads=1, head_dim=64)
    q, at = _bf16(rng, 2 * new, 4, 64).cuda(), _ids(0, new, 2 * new)
    want = cache.attend(0, q, _ids(0, 1), at, max_new=new)
    for kw in (dict(window=1 << 32), dict(window=(1 << 31) - 1, sinks=1 << 40), dict(window=1, sinks=(1 << 32) - 1),
               dict(window=(1 << 32) + 1, max_len=1 << 32)):
        got = cache.attend(0, q, _ids(0, 1), at, max_new=new, **kw)
        cache.check()
        # the tiles may be dealt to workgroups in another way, so sums may round otherwise
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max()), kw


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 65, 128, 129, 192, 200, 256])
def test_many_rows_split_and_joined(dim, dtype):
    """Prompts long enough for several splits, at head sizes of every width of the join."""
    print("split prompts", dim, dtype, flush=True)
    rng = np.random.default_rng(dim)
    lens, new, heads = [3000, 700], [70, 90], 3
    cache, model = _filled(rng, lens, kv_heads=1, head_dim=dim, dtype=dtype)
    at = [0, 70, 160]
    q = _bf16(rng, 160, heads, dim)
    for kw in ({}, dict(window=1500, sinks=3), dict(softcap=30.0)):
        cache._attend_work = None
        got, lse = cache.attend(0, q.cuda(), _ids(0, 1), _ids(*at), max_new=90, lse=True, **kw)
        cache.check()
        assert cache._attend_work.numel() >= 4 * 160 * heads * 2 * (-(-dim // 64) * 64 + 4), "not split"
        out, ref, slack, spread = model.attend(0, _f64(q), [0, 1], at, **kw)
        assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread)), float(np.abs(_f64(got) - out).max())
        assert np.all(np.abs(_f64(lse) - ref) <= slack + 2.0 ** -20 * (1 + np.abs(ref)))


def _bits(cache):
    torch.cuda.synchronize()
    return {n: getattr(cache, n).clone().view(torch.uint8).cpu() for n in ("k", "v", "scale", "refs", "table", "lens")}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dim,page", [(64, 16), (80, 32), (256, 128)])
def test_refused_appends_write_nothing(dim, page, f32):
    """Token ranges, rows and table entries that do not exist: no byte of the
    cache changes but those of the good rows' own pages, which get the data
    that they hold already."""
    rng = np.random.default_rng(dim)
    kw = dict(layers=2, kv_heads=2, head_dim=dim, n_pages=12, max_seqs=3, max_pages=6, page_tokens=page, dtype="e4m3")
    cache = kv.KvCache(**kw)
    for n in ("k", "v"):
        t = getattr(cache, n)
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
    cache.scale.fill_(float("nan"))
    cache.extend(_ids(1, 2), _ids(20, 10))
    x = _bf16(rng, 40, 2, dim).cuda()
    x = x.float() * 1.001 if f32 else x
    cache.append(1, x[:30], x[:30], _ids(1, 2), _ids(0, 20, 30))
    cache.check()
    before = _bits(cache)
    for rows, starts in (((1, 0), (0, 21, 30)), ((1, 0), (0, 20, 31)), ((1, 0), (5, 0, 30)), ((1, 0), (-1, 19, 29)),
                         ((3, -1), (0, 1, 2)), ((1 << 30, 0), (0, 1, 1)), ((1, 2), (0, 20, 31)), ((1, 2), (0, 20, 41))):
        cache.append(1, x, x, _ids(*rows), _ids(*starts))
        with pytest.raises(RuntimeError, match="does not exist"):
            cache.check()
        after = _bits(cache)
        assert all(torch.equal(before[n], after[n]) for n in before), (rows, starts)
    for entry in (-5, -1, 12, 1 << 30, -(1 << 31)):
        own = cache.table[1].clone()
        last = (20 - 1) // page
        cache.table[1, last] = entry
        before = _bits(cache)
        cache.append(1, x[19:31], x[19:31], _ids(1, 2), _ids(0, 1, 11))      # the good row's own data again
        if entry == 12:
            cache.append(0, x[:20], x[:20], _ids(1), _ids(0, 20), max_new=20)
        with pytest.raises(RuntimeError, match="does not exist"):
            cache.check()
        good = set() if entry != 12 else {(0, int(p)) for p in own[:last]}   # whole pages before the bad one
        after = _bits(cache)
        for n in ("k", "v", "scale"):
            same = (before[n] == after[n]).flatten(2).all(dim=2)
            for layer, p in good:
                same[layer, p] = True
            assert bool(same.all()), (entry, n)
        assert all(torch.equal(before[n], after[n]) for n in ("refs", "table", "lens"))
        cache.table[1].copy_(own)


def test_two_threads_over_one_cache():
    """Attention, adapters and pages from threads that share a cache, a pack and a stream."""
    import threading
    from lossless_entropy_coding_amd import lora
    rng = np.random.default_rng(51)
    cache, _ = _filled(rng, [3000, 500, 90, 40], kv_heads=1, head_dim=64)
    pack = lora.LoraPack([(_bf16(rng, 16, 96), _bf16(rng, 40, 16), 0.5)])
    work = []
    for i in range(4):
        n = 1 + i
        q, rows = _bf16(rng, 64 * n, 8, 64).cuda(), _ids(*range(n))
        at = _ids(*range(0, 64 * n + 1, 64))
        x, batch = _bf16(rng, 30 + i, 96).cuda(), lora.LoraBatch(torch.zeros(30 + i, dtype=torch.int32, device="cuda"), 1)
        y = torch.zeros(30 + i, 40, device="cuda")
        call = lambda q=q, rows=rows, at=at, x=x, batch=batch, y=y: (   # noqa: E731
            cache.attend(0, q, rows, at, max_new=64), pack.add(y, x, batch, out=torch.empty_like(y)))
        work.append((call, call()))
    torch.cuda.synchronize()
    wrong = []

    def go(call, want):
        for _ in range(50):
            got = call()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                wrong.append(1)
    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    cache.check()


@pytest.mark.parametrize("new,dim,heads,dtype", [(1, 64, 4, "int8"), (1, 256, 2, "e4m3"), (3, 128, 20, "e4m3"), (15, 80, 4, "int8"),
                                                 (1, 192, 63, "e4m3")])
def test_few_rows_hold_probabilities_in_16_bits(new, dim, heads, dtype):
    """Values of either sign that nearly cancel: a probability's error shows
    beside the result's own rounding.  Each part of P is rounded by at most
    2^-8 of it (8 significant bits), the two by 2^-16; its product with a code
    is exact; fp32 sums are in the logits' slack, which counts twice."""
    print("probabilities", new, dim, heads, dtype, flush=True)
    rng = np.random.default_rng(dim + heads)
    lens = [5000, 70, 1]
    cache, model = _filled(rng, lens, kv_heads=1, head_dim=dim, dtype=dtype)
    q = _bf16(rng, 3 * new, heads, dim)
    at = [0, new, 2 * new, 3 * new]
    for kw in ({}, dict(window=700, sinks=4), dict(softcap=30.0)):
        got = cache.attend(0, q.cuda(), _ids(0, 1, 2), _ids(*at), max_new=new, **kw)
        cache.check()
        out, ref, slack, spread = model.attend(0, _f64(q), [0, 1, 2], at, **kw)
        slack = np.where(np.isneginf(ref), 0, slack)
        bound = (2.0 ** -16 + 2.02 * slack[..., None]) * spread + 2.0 ** -8 * 1.01 * np.abs(out) + 1e-30
        assert np.all(np.abs(_f64(got) - out) <= bound), (kw, float((np.abs(_f64(got) - out) / bound).max()))


@pytest.mark.parametrize("cap", [30.0, 300.0])
@pytest.mark.parametrize("new,dim", [(1, 64), (70, 128), (70, 256)])
def test_capped_logits_of_an_infinite_query(new, dim, cap):
    """Keys that are positive in every channel times an infinity are infinite,
    capped to c, and so all alike: the result is the mean of the values."""
    rng = np.random.default_rng(dim)
    lens = [300, 90]
    cache, model = _filled(rng, lens, kv_heads=1, head_dim=dim)
    k = _bf16(rng, sum(lens), 1, dim).abs() + 0.5
    v = _bf16(rng, sum(lens), 1, dim)
    cache.append(0, k.cuda(), v.cuda(), _ids(0, 1), _ids(0, 300, 390))
    model.append(0, _f64(k), _f64(v), [0, 1], [0, 300, 390])
    q = _bf16(rng, 2 * new, 2, dim)
    q[:, 0, 3], q[:, 1, dim - 1] = float("inf"), float("-inf")
    got, lse = cache.attend(0, q.cuda(), _ids(0, 1), _ids(0, new, 2 * new), max_new=new, softcap=cap, lse=True)
    cache.check()
    for r, n in enumerate(lens):
        values = model.tokens(0, r, 0, 1)
        for j in range(new):
            see = n - new + j + 1
            want, spread = values[:see].mean(axis=0), np.abs(values[:see]).mean(axis=0)
            for h, sign in ((0, 1), (1, -1)):
                bound = (2.0 ** -8 * 1.01 + 2.0 ** -14) * spread + 2.0 ** -8 * 1.01 * np.abs(want)
                assert np.all(np.abs(_f64(got[r * new + j, h]) - want) <= bound), (r, j, h)
                assert abs(float(lse[r * new + j, h]) - (sign * cap + np.log(see))) <= 2.0 ** -20 * (cap + 10)
