"""Attention of rows that share their first tokens, on the GPU against the
cache's plain model (oracle.serving.Cache.attend) within the bound that
oracle.serving.attend_bound derives."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from oracle import serving as S
from test_gpu_kv import _bf16, _f64, _fill, _ids, _pair

pytestmark = pytest.mark.gpu


def _branch(rng, page, dim, kv_heads, dtype, groups, common, own, size=1.0, spare=1, layers=1):
    """groups[g] rows that go on from common[g] tokens, each by up to `own` more; rows in any order.  The pool's bytes are
    stale and its scales NaN where nothing was stored."""
    n = sum(groups)
    most = -(-(max(common) + own) // page) + 3
    cache, model = _pair(layers=layers, kv_heads=kv_heads, head_dim=dim, n_pages=n * (-(-own // page) + 5) + len(groups) * most + 3,
                         max_seqs=n + spare, max_pages=most, page_tokens=page, dtype=dtype)
    order = [int(r) for r in rng.permutation(n + spare)[:n]]
    at = 0
    for rows, tokens in zip(groups, common):
        mine = order[at:at + rows]
        at += rows
        if tokens and rows:
            _fill(cache, model, rng, mine[:1], [tokens], (size,))
            if rows > 1:
                for c in (cache, model):
                    ids = _ids if c is cache else lambda *v: list(v)
                    c.fork(ids(*[mine[0]] * (rows - 1)), ids(*mine[1:]))
    more = [int(x) for x in rng.integers(0, own + 1, n)]
    if own:
        more[0] = own
        _fill(cache, model, rng, order, more, (size,))
    assert model.status == 0
    return cache, model, order, more


def _check(cache, model, rng, rows, counts, groups, heads, layer=0, size=1.0, gone=(), flags=0, **kw):
    total = sum(counts)
    q = _bf16(rng, total, heads, cache.head_dim, size=size)
    offs = [0] + [int(x) for x in np.cumsum(groups)]
    b = kv.KvBatch(cache, _ids(*rows), _ids(*counts), groups=_ids(*offs), total=total, max_new=max(counts),
                   max_len=kw.pop("max_len", 0))
    got, lse = cache.attend_shared(layer, q.cuda(), b, lse=True, **kw)
    again, lse2 = cache.attend_shared(layer, q.cuda(), b, lse=True, **kw)
    starts = [0] + [int(x) for x in np.cumsum(counts)]
    out, ref, slack, spread = model.attend(layer, _f64(q), rows, starts, gone=gone, **kw)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == flags
    assert torch.equal(got, again) and torch.equal(lse, lse2)
    g, l = _f64(got), _f64(lse)
    empty = np.isneginf(ref)
    assert np.array_equal(empty, np.isneginf(l)) and np.all(g[empty] == 0)
    off = np.abs(g - out) / S.attend_bound(out, slack, spread)
    assert np.all(off <= 1), float(off.max())
    assert np.all(np.abs(l - ref)[~empty] <= slack[~empty] + 2.0 ** -20 * (1 + np.abs(ref[~empty])))
    return q, b, got, lse


SHAPES = [  # head_dim, page, kv_heads, heads, rows of the groups, their common tokens, own tokens
    (64, 16, 1, 1, [1], [1], 0),
    (64, 16, 1, 1, [2], [64], 1),
    (128, 64, 2, 4, [5], [700], 60),
    (128, 16, 1, 5, [9, 1, 3], [130, 2000, 63], 200),
    (256, 16, 2, 4, [4], [600], 24),
    (256, 64, 1, 2, [40], [1300], 130),
    (192, 32, 1, 3, [7, 8], [900, 0], 70),
    (80, 32, 3, 3, [17], [257], 33),
    (1, 16, 1, 2, [3], [100], 5),
    (72, 256, 1, 7, [6], [1000], 300),
    (128, 128, 1, 8, [1, 1, 1], [3000, 64, 128], 1),
    (96, 16, 4, 16, [70], [64], 2),
]


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page,kv_heads,heads,groups,common,own", SHAPES)
def test_single_tokens_of_groups(dtype, dim, page, kv_heads, heads, groups, common, own):
    print("shared", dtype, dim, page, kv_heads, heads, groups, common, own, flush=True)
    rng = np.random.default_rng(dim + page + sum(groups))
    cache, model, rows, _ = _branch(rng, page, dim, kv_heads, dtype, groups, common, own)
    ones = [1] * len(rows)
    for kw in ({}, dict(window=5), dict(window=200, sinks=3), dict(softcap=20.0), dict(scale=-0.3),
               dict(window=1, sinks=200, softcap=50.0), dict(max_len=int(model.lens.max())), dict(softcap=1000.0, window=90)):
        _check(cache, model, rng, rows, ones, groups, heads, **kw)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page,kv_heads,heads,groups,common,own,most", [
    (64, 16, 1, 1, [3], [100], 50, 30), (128, 32, 2, 10, [4, 2], [400, 70], 20, 4), (256, 64, 1, 2, [6], [500], 40, 31),
    (96, 16, 1, 5, [3, 3], [64, 300], 0, 12), (128, 16, 1, 4, [2], [300], 90, 16), (256, 16, 1, 2, [3], [200], 60, 50)])
def test_several_tokens_of_a_row(dtype, dim, page, kv_heads, heads, groups, common, own, most):
    """Drafts and chunks, some of whose tokens are among the common ones, rows without any; the last two have 64 stacked
    rows and more."""
    rng = np.random.default_rng(dim + most)
    cache, model, rows, _ = _branch(rng, page, dim, kv_heads, dtype, groups, common, own)
    counts = [int(min(c, model.lens[r])) for r, c in zip(rows, rng.integers(0, most + 1, len(rows)))]
    counts[0] = int(min(most, model.lens[rows[0]]))
    for kw in ({}, dict(window=33, sinks=2), dict(softcap=30.0), dict(window=1)):
        _check(cache, model, rng, rows, counts, groups, heads, **kw)


def test_long_common_tokens_are_split():
    rng = np.random.default_rng(2)
    for dim, kv_heads, heads, groups, common, own, dtype in ((128, 1, 5, [8], [30000], 700, "e4m3"), (64, 2, 2, [2, 1], [9000, 20000], 5000, "int8")):
        cache, model, rows, _ = _branch(rng, 32, dim, kv_heads, dtype, groups, common, own)
        for kw in ({}, dict(window=8000, sinks=70), dict(max_len=int(model.lens.max()))):
            _check(cache, model, rng, rows, [1] * len(rows), groups, heads, **kw)


def test_large_logits_and_far_apart_scales():
    rng = np.random.default_rng(8)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [6], [300], 100, size=12.0)
    _fill(cache, model, rng, rows, [17] * 6, (1e-4,))
    _check(cache, model, rng, rows, [1] * 6, [6], 3, size=6.0)


def test_it_is_attend():
    """On the same rows: equal to rounding, both within 16-bit probabilities of the exact result."""
    rng = np.random.default_rng(5)
    cache, model, rows, _ = _branch(rng, 64, 128, 2, "int8", [20], [900], 200)
    q, b, got, lse = _check(cache, model, rng, rows, [1] * 20, [20], 10)
    want, wlse = cache.attend(0, q.cuda(), _ids(*rows), lse=True)
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    assert (lse - wlse).abs().max() <= 2.0 ** -18 * (1 + wlse.abs().max())


@pytest.mark.parametrize("dim,dtype", [(64, "e4m3"), (128, "int8"), (256, "e4m3")])
def test_probabilities_have_16_bits(dim, dtype):
    """The error over the result's own rounding is that of fp32 sums: 2^-15 of the values' spread covers 16 significant
    bits (2^-17 of each term) and logits moved by `slack`."""
    rng = np.random.default_rng(dim)
    cache, model, rows, _ = _branch(rng, 64, dim, 1, dtype, [24], [1500], 100)
    q, b, got, lse = _check(cache, model, rng, rows, [1] * 24, [24], 2)
    out, ref, slack, spread = model.attend(0, _f64(q), rows)
    bound = (2.0 ** -15 + 2.02 * slack[..., None]) * spread + 2.0 ** -9 * 1.01 * np.abs(out) * 2
    assert np.all(np.abs(_f64(got) - out) <= bound)


def test_rows_that_see_nothing_and_tokens_of_no_row():
    """Empty rows, more new tokens than a row holds, tokens behind the last row, which are left as they were."""
    rng = np.random.default_rng(6)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [3], [100], 10, spare=2)
    empty = [r for r in range(5) if model.lens[r] == 0]
    use = [rows[0], empty[0], rows[1]]
    q = _bf16(rng, 8, 2, 64)
    b = kv.KvBatch(cache, _ids(*use), _ids(1, 1, 2), total=8, max_new=3)       # four tokens of no row
    out, lse = torch.full((8, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, 2), 5.0, device="cuda")
    cache.attend_shared(0, q.cuda(), b, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 4                                        # the plan said so
    cache.status.zero_()
    assert (out[4:] == 3).all() and (lse[4:] == 5).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    want, ref, slack, spread = model.attend(0, _f64(q)[:4], use, [0, 1, 2, 4])
    assert np.all(np.abs(_f64(out[:4]) - want) <= S.attend_bound(want, slack, spread))
    none = cache.attend_shared(0, q[:0].cuda(), kv.KvBatch(cache, _ids(), total=0))
    assert none.shape == (0, 2, 64)
    none = cache.attend_shared(0, q[:0].cuda(), kv.KvBatch(cache, _ids(*use), _ids(0, 0, 0), total=0))
    assert none.shape == (0, 2, 64)
    cache.check()


def test_groups_that_have_nothing_in_common_and_rows_of_no_group():
    rng = np.random.default_rng(7)
    cache, model, rows, _ = _branch(rng, 16, 128, 1, "int8", [1, 1, 1, 1, 3], [500, 64, 300, 10, 200], 40)
    ones = [1] * 7
    _check(cache, model, rng, rows, ones, [7], 4)                  # one group, no common pages
    _check(cache, model, rng, rows, ones, [4, 3], 4)
    _check(cache, model, rng, rows, ones, [0, 5, 0, 2, 0], 4)      # empty groups, a family cut in two
    q = _bf16(rng, 7, 4, 128)
    for offs in ([2, 5], [0], [7, 7], [4, 7]):
        b = kv.KvBatch(cache, _ids(*rows), groups=_ids(*offs))
        got = cache.attend_shared(0, q.cuda(), b)
        out, _, slack, spread = model.attend(0, _f64(q), rows)
        assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread)), offs
    b = kv.KvBatch(cache, _ids(rows[4], rows[4], rows[5], rows[4]))          # a row named more than once
    got = cache.attend_shared(0, q[:4].cuda(), b)
    out, _, slack, spread = model.attend(0, _f64(q[:4]), [rows[4], rows[4], rows[5], rows[4]])
    assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))
    cache.check()


@pytest.mark.parametrize("dim,dtype", [(64, "int8"), (256, "e4m3")])
def test_queries_that_are_not_finite(dim, dtype):
    """A NaN in a query gives NaN twice in its row and head, and nowhere else."""
    rng = np.random.default_rng(9)
    cache, model, rows, _ = _branch(rng, 16, dim, 1, dtype, [20], [200], 30)
    q = _bf16(rng, 20, 2, dim)
    bad = [(3, 0), (17, 1)]
    q[3, 0, 5] = float("nan")
    q[17, 1, 0] = float("nan")
    got, lse = cache.attend_shared(0, q.cuda(), kv.KvBatch(cache, _ids(*rows)), lse=True)
    for t, h in bad:
        assert got[t, h].isnan().all() and lse[t, h].isnan()
        q[t, h] = 0
        got[t, h] = lse[t, h] = 0
    assert got.isfinite().all() and lse.isfinite().all()
    out, ref, slack, spread = model.attend(0, _f64(q), rows)
    for t, h in bad:
        out[t, h] = 0
    assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))


def test_tokens_without_a_page_are_left_out():
    """Entries of the table that name no page after the plan was made: reported, and their tokens left out."""
    rng = np.random.default_rng(10)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [5], [400], 100)
    q = _bf16(rng, 5, 2, 64)
    b = kv.KvBatch(cache, _ids(*rows))
    own = int(b.shared[0]) // 16 + 1
    cache.table[rows[0], 3] = 1 << 30                              # a common page, of the group's first row
    cache.table[rows[1], own] = -5                                 # a page of a row's own
    got, lse = cache.attend_shared(0, q.cuda(), b, lse=True)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 4
    gone = [(r, 3) for r in rows] + [(rows[1], own)]
    out, ref, slack, spread = model.attend(0, _f64(q), rows, gone=gone)
    assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))
    assert np.all(np.abs(_f64(lse) - ref) <= slack + 2.0 ** -20 * (1 + np.abs(ref)))


def test_plans_that_no_longer_hold_read_nothing_out_of_range():
    """Rows freed, or never there, after the plan: places and pages are bounded by the cache, whatever the results are."""
    rng = np.random.default_rng(11)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "int8", [4], [300], 60)
    q = _bf16(rng, 4, 2, 64).cuda()
    b = kv.KvBatch(cache, _ids(*rows))
    cache.free(_ids(*rows))
    cache.attend_shared(0, q, b)
    for value in (1 << 30, -5):
        b.update(_ids(*rows))
        b.places.fill_(value)
        cache.attend_shared(0, q, b)
    for word in range(6):
        for value in (77, 1 << 20, 1 << 30, -9):
            b.update(_ids(*rows))
            b._info[4:].view(-1, 8)[:, word] = value
            cache.attend_shared(0, q, b)
    torch.cuda.synchronize()


def test_strided_queries_and_results():
    rng = np.random.default_rng(12)
    cache, model, rows, _ = _branch(rng, 16, 72, 1, "e4m3", [9], [200], 30)
    b = kv.KvBatch(cache, _ids(*rows))
    for pad in (0, 1, 4, 8):
        wide = torch.zeros(9, 3 * 72 + pad, dtype=torch.bfloat16, device="cuda")
        q = wide.as_strided((9, 3, 72), (3 * 72 + pad, 72, 1))
        q.copy_(_bf16(rng, 9, 3, 72))
        flat = torch.full((9 * (3 * 72 + pad) + 3,), 2.0, dtype=torch.bfloat16, device="cuda")
        o = flat[3 if pad == 1 else 0:].as_strided((9, 3, 72), (3 * 72 + pad, 72, 1))
        cache.attend_shared(0, q, b, out=o)
        want, _, slack, spread = model.attend(0, _f64(q), rows)
        assert np.all(np.abs(_f64(o) - want) <= S.attend_bound(want, slack, spread))
        assert int((flat == 2.0).sum()) >= flat.numel() - 9 * 3 * 72
    cache.check()


def test_a_search_in_a_graph():
    """A captured step (plan, append, attention of every layer) of a beam search, replayed with eager moves of the rows in
    between; another captured step shares its workspace."""
    rng = np.random.default_rng(13)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [6], [150], 20, layers=2)
    ids, ones, n = _ids(*rows), _ids(*[1] * 6), 6
    k, v = (torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    b = kv.KvBatch(cache, ids)

    def step():
        cache.extend(ids, ones)
        b.update(ids)
        got = []
        for layer in range(2):
            cache.append(layer, k, v, ids)
            got.append(cache.attend_shared(layer, q, b))
        return got
    cache.attend_shared(0, q, b)                                   # the workspace
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                got = step()
            graphs.append((g, got))
    torch.cuda.current_stream().wait_stream(side)
    for i in range(6):
        x = [_bf16(rng, n, 1, 64) for _ in range(2)] + [_bf16(rng, n, 2, 64)]
        for to, t in zip((k, v, q), x):
            to.copy_(t)
        g, got = graphs[i % 2]
        g.replay()
        model.extend(rows, [1] * n)
        for layer in range(2):
            model.append(layer, _f64(x[0]), _f64(x[1]), rows)
        for layer in range(2):
            out, _, slack, spread = model.attend(layer, _f64(x[2]), rows)
            assert np.all(np.abs(_f64(got[layer]) - out) <= S.attend_bound(out, slack, spread)), (i, layer)
        parents = [int(p) for p in rng.integers(0, n, n)]
        cache.reorder(ids, _ids(*parents))
        model.reorder(rows, parents)
        assert cache.table.cpu().numpy().tobytes() == model.table.tobytes()
    cache.check()


def test_work_on_another_stream():
    rng = np.random.default_rng(14)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [6], [150], 20)
    q = _bf16(rng, 6, 2, 64).cuda()
    want = cache.attend_shared(0, q, kv.KvBatch(cache, _ids(*rows)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros(64 << 20, device="cuda")
    for _ in range(5):
        busy.add_(1)
    b = kv.KvBatch(cache, _ids(*rows), stream=side)
    got = cache.attend_shared(0, q, b, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
