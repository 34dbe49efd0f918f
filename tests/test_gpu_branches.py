"""Rows that branch from common tokens, on the GPU against the cache's plain
model (oracle.serving.Cache): the move of rows to their parents and the plan of
a step's tokens, both equal bit for bit."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from test_gpu_kv import _fill, _ids, _pair, _same

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- reorder
@pytest.mark.parametrize("seed,page,layers,dim", [(0, 16, 2, 24), (1, 32, 1, 64), (2, 16, 3, 100), (3, 64, 2, 16), (4, 128, 1, 8)])
def test_rows_follow_their_parents(seed, page, layers, dim):
    """Random growth, forks, moves and frees of a small pool; every buffer after every call."""
    rng = np.random.default_rng(seed)
    cache, model = _pair(layers=layers, kv_heads=2, head_dim=dim, n_pages=60, max_seqs=12, max_pages=9, page_tokens=page, dtype="int8")
    refused = 0
    for step in range(60):
        op = rng.choice(["extend", "fork", "reorder", "reorder", "reorder", "free"])
        used = [r for r in range(12) if model.lens[r]]
        empty = [r for r in range(12) if not model.lens[r]]
        print("step", step, op, flush=True)
        if op == "extend":
            rows = [int(r) for r in rng.permutation(12)[:rng.integers(1, 6)]]
            counts = [int(c) for c in rng.integers(0, 2 * page, len(rows))]
            cache.extend(_ids(*rows), _ids(*counts))
            model.extend(rows, counts)
        elif op == "fork" and used and empty:
            kids = empty[:rng.integers(1, len(empty) + 1)]
            parents = [int(rng.choice(used)) for _ in kids]
            cache.fork(_ids(*parents), _ids(*kids))
            model.fork(parents, kids)
        elif op == "free" and len(used) > 6:
            cache.free(_ids(used[0]))
            model.free(used[:1])
        elif op == "reorder":
            rows = [int(r) for r in rng.permutation(12)[:rng.integers(1, 13)]]
            parents = [int(q) for q in rng.integers(-1 if rng.random() < 0.3 else 0, len(rows), len(rows))]
            if rng.random() < 0.2:
                parents = [int(q) for q in rng.permutation(len(rows))]           # a permutation: no copies
            before = model.status
            cache.reorder(_ids(*rows), _ids(*parents))
            model.reorder(rows, parents)
            refused += model.status != before
        _same(cache, model)
        if model.status:
            cache.status.zero_()
            model.status = 0
    assert int(model.refs.sum()) == sum(model.pages(n) for n in model.lens)


@pytest.mark.parametrize("n,max_pages,page", [(1, 5, 16), (7, 300, 16), (64, 70, 32), (700, 9, 16), (4096, 3, 16)])
def test_numbers_of_rows(n, max_pages, page):
    """Columns of the table in every width that a workgroup takes."""
    rng = np.random.default_rng(n)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=8, n_pages=n * min(max_pages, 40) + n + 5, max_seqs=n + 2, max_pages=max_pages,
                         page_tokens=page, dtype="e4m3")
    rows = [int(r) for r in rng.permutation(n + 2)[:n]]
    counts = [int(c) for c in rng.integers(0, min(max_pages, 39) * page, n)]
    if n == 7:
        counts[3] = 38 * page + 1
    for call in (cache, model):
        ids = _ids if call is cache else lambda *v: list(v)
        call.extend(ids(*rows), ids(*counts))
    for _ in range(3):
        parents = [int(q) for q in rng.integers(0, n, n)]
        cache.reorder(_ids(*rows), _ids(*parents))
        model.reorder(rows, parents)
        _same(cache, model)
        assert model.status == 0


def test_moves_that_are_refused_change_nothing():
    cache, model = _pair(layers=1, kv_heads=1, head_dim=16, n_pages=7, max_seqs=5, max_pages=4, page_tokens=16, dtype="e4m3")
    rng = np.random.default_rng(1)
    _fill(cache, model, rng, [0, 1, 2], [20, 17, 16])            # 2 + 2 + 1 pages, two are free

    def refused(bit, rows, parents):
        cache.reorder(_ids(*rows), _ids(*parents))
        model.status |= bit
        _same(cache, model)
        cache.status.zero_()
        model.status = 0
    refused(1, [0, 1, 2, 3], [0, 0, 0, 0])                       # three copies, two free pages
    refused(4, [0, 5], [0, 0])                                   # no row 5
    refused(4, [0, -1], [0, 0])
    refused(4, [0, 1], [0, 2])                                   # no parent 2
    refused(4, [0, 1], [0, -2])
    refused(4, [0, 1, 0], [0, 1, 2])                             # a row named twice
    cache.lens[1] = 65
    cache.reorder(_ids(0, 1), _ids(1, 1))                        # longer than its row of the table
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 2 and cache.lens.tolist() == [20, 65, 16, 0, 0]
    cache.status.zero_()
    cache.lens[1] = 17
    at = cache.table[0, 1].clone()
    cache.table[0, 1] = 1 << 30                                  # the page to be copied does not exist
    cache.reorder(_ids(0, 1), _ids(0, 0))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 4
    cache.table[0, 1] = at
    cache.status.zero_()
    _same(cache, model)
    cache.reorder(_ids(0, 1), _ids(0, 0))                        # what was free is enough
    model.reorder([0, 1], [0, 0])
    _same(cache, model)
    cache.reorder(_ids(0, 1, 2), _ids(-1, -1, -1))
    model.reorder([0, 1, 2], [-1, -1, -1])
    _same(cache, model)
    assert int(cache.refs.sum()) == 0
    with pytest.raises(Exception, match="at most 4096"):
        cache.reorder(torch.zeros(4097, dtype=torch.int32, device="cuda"), torch.zeros(4097, dtype=torch.int32, device="cuda"))


def test_bad_entries_of_whole_pages_are_reported():
    cache, model = _pair(layers=1, kv_heads=1, head_dim=16, n_pages=9, max_seqs=3, max_pages=4, page_tokens=16, dtype="e4m3")
    cache.extend(_ids(0, 1), _ids(40, 16))
    cache.table[0, 0] = -7
    cache.reorder(_ids(0, 1), _ids(0, 0))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 4 and cache.lens.tolist() == [40, 40, 0]
    assert cache.table[1, 0] == -7 and int(cache.refs.max()) == 2


def test_a_captured_move_replays():
    cache, model = _pair(layers=2, kv_heads=1, head_dim=32, n_pages=40, max_seqs=4, max_pages=8, page_tokens=16, dtype="int8")
    rng = np.random.default_rng(3)
    _fill(cache, model, rng, [0, 1, 2, 3], [50, 33, 16, 60])
    rows, parents = _ids(0, 1, 2, 3), _ids(0, 1, 2, 3)
    cache.reorder(rows, parents)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.reorder(rows, parents)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(5):
        p = [int(q) for q in rng.integers(0, 4, 4)]
        parents.copy_(_ids(*p))
        graph.replay()
        model.reorder([0, 1, 2, 3], p)
        _same(cache, model)
        _fill(cache, model, rng, [0, 1, 2, 3], [3, 1, 2, 3])
        _same(cache, model)


# --------------------------------------------------------------------- plans
def _plan_same(b, want):
    for name, w in zip(("starts", "places", "slots", "table", "lead", "shared"), want):
        np.testing.assert_array_equal(getattr(b, name).cpu().numpy(), w, err_msg=name)
    assert int(b._info[0]) == 0


def _branched(seed, page, groups, rows, common, own):
    """`groups` of rows that share their first tokens' pages, then grow by up to `own` tokens each, on rows in any order."""
    rng = np.random.default_rng(seed)
    n, most = groups * rows, -(-(common + own + 1) // page) + 1
    cache, model = _pair(layers=1, kv_heads=1, head_dim=8, n_pages=n * most, max_seqs=n + 1, max_pages=most, page_tokens=page, dtype="int8")
    order = [int(r) for r in rng.permutation(n + 1)[:n]]
    for g in range(groups):
        mine = order[g * rows:(g + 1) * rows]
        for c in (cache, model):
            ids = _ids if c is cache else lambda *v: list(v)
            c.extend(ids(mine[0]), ids(common + 7 * g))
            if rows > 1:
                c.fork(ids(*[mine[0]] * (rows - 1)), ids(*mine[1:]))
    more = [int(x) for x in rng.integers(0, own + 1, n)]
    cache.extend(_ids(*order), _ids(*more))
    model.extend(order, more)
    assert model.status == 0
    return rng, cache, model, order


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("groups,rows,common,own", [(1, 1, 40, 3), (1, 5, 300, 40), (4, 3, 130, 500), (3, 70, 65, 9), (1, 300, 513, 20)])
def test_plans(page, groups, rows, common, own):
    rng, cache, model, order = _branched(page + rows, page, groups, rows, common, own)
    offs = [g * rows for g in range(groups + 1)]
    counts = [int(min(c, model.lens[r])) for r, c in zip(order, rng.integers(0, 30, len(order)))]
    longest = int(model.lens.max())
    b = kv.KvBatch(cache, _ids(*order), _ids(*counts), groups=_ids(*offs), total=sum(counts), max_len=longest)
    _plan_same(b, model.batch(order, counts, offs, sum(counts), -(-longest // page)))
    assert (b.shared >= common // page * page // 64 * 64).all()
    b = kv.KvBatch(cache, _ids(*order))                          # a token each, one group
    _plan_same(b, model.batch(order, [1] * len(order), [0, len(order)], len(order), cache.max_pages))
    offs = sorted(int(x) for x in rng.integers(0, len(order) + 1, 6))       # empty groups, rows of none
    b = kv.KvBatch(cache, _ids(*order), groups=_ids(*offs))
    _plan_same(b, model.batch(order, [1] * len(order), offs, len(order), cache.max_pages))
    cache.check()


def test_long_rows_and_many_new_tokens():
    """More tokens and pages than a workgroup takes at a time."""
    rng, cache, model, order = _branched(9, 16, 1, 3, 60000, 9000)
    counts = [int(model.lens[r]) - 60000 for r in order]
    counts[0] = int(model.lens[order[0]])
    b = kv.KvBatch(cache, _ids(*order), _ids(*counts), total=sum(counts))
    _plan_same(b, model.batch(order, counts, [0, 3], sum(counts), cache.max_pages))
    one = order[1]
    at = 3000
    cache.table[one, at] = model.table[one, at] = model.table[one, at + 1]  # rows part on the way
    b.update(_ids(*order), _ids(*counts))
    _plan_same(b, model.batch(order, counts, [0, 3], sum(counts), cache.max_pages))
    assert b.shared[1] == at * 16 // 64 * 64


def test_plans_of_bad_rows_counts_and_groups():
    _, cache, model, order = _branched(5, 16, 1, 4, 100, 10)
    n = 4

    def flagged(rows, counts, groups, total, **kw):
        b = kv.KvBatch(cache, _ids(*rows), _ids(*counts), groups=None if groups is None else _ids(*groups), total=total, **kw)
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 4
        cache.status.zero_()
        return b
    b = flagged([order[0], 77, order[2], -1], [1, 1, 1, 1], None, 4)
    assert b.places.tolist()[1] == -1 and b.slots.tolist()[3] == -1 and (b.table[1] == -1).all() and (b.shared == 0).all()
    b = flagged(order, [1, -3, 2, 1], None, 4)
    assert b.starts.tolist() == [0, 1, 1, 3, 4]
    b = flagged(order, [1, 500, 1, 1], None, 503)                # more than the row holds
    assert (b.places[1:300] == -1).all() and int(b.places[500]) == int(cache.lens[order[1]]) - 1
    b = flagged(order, [2, 2, 2, 2], None, 7)
    assert b.starts.tolist() == [0, 2, 4, 6, 7]
    b = flagged(order, [2, 2, 2, 2], None, 9)
    assert b.places[8] == -1 and b.slots[8] == -1
    flagged(order, [2, 2, 2, 2], None, 8, max_new=1)
    b = flagged(order, [1] * 4, [0, 3, 2, 4], 4)
    b = flagged(order, [1] * 4, [-5, 2, 9], 4)
    assert b.lead.tolist()[0] == 0
    cache.table[order[1], 2] = -1
    b = flagged(order, [100] * 4, None, 400)                     # a page that does not exist
    assert (b.shared == 0).all()
    b = kv.KvBatch(cache, _ids(), _ids(), total=0)
    assert b.starts.numel() == 1
    cache.check()
    assert n == 4


def test_a_captured_plan_replays():
    rng, cache, model, order = _branched(6, 16, 2, 4, 200, 60)
    rows, counts, offs = _ids(*order), _ids(*[1] * 8), _ids(0, 4, 8)
    b = kv.KvBatch(cache, rows, counts, groups=offs, total=8, max_new=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.update(rows, counts, groups=offs)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        order = [order[int(i)] for i in rng.permutation(8)]
        c = [0, 2, 0, 1, 3, 1, 0, 1]
        rng.shuffle(c)
        rows.copy_(_ids(*order))
        counts.copy_(_ids(*c))
        graph.replay()
        _plan_same(b, model.batch(order, [int(x) for x in c], [0, 4, 8], 8, cache.max_pages))
        kv.KvBatch(cache, rows[:3].contiguous())
    cache.check()
