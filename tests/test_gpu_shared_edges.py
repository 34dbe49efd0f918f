"""Corners of the attention of groups, on the GPU."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import beam, kv
from oracle import serving as S
from test_gpu_beam import _check as _choices
from test_gpu_kv import _bf16, _f64, _fill, _ids, _same
from test_gpu_shared import _branch, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,heads,own", [(64, 2, 200), (256, 3, 90), (128, 4, 3000)])
def test_rows_of_no_groups(dim, heads, own):
    """Offsets of no groups: every row by itself, whole and split."""
    rng = np.random.default_rng(dim)
    cache, model, rows, _ = _branch(rng, 16, dim, 1, "int8", [3, 1, 5], [100, 70, 300], own)
    _check(cache, model, rng, rows, [1] * 9, [], heads)
    _check(cache, model, rng, rows, [1, 0, 2, 1, 3, 1, 1, 0, 2], [], heads, window=50, sinks=2)


@pytest.mark.parametrize("common", [700, 30000])
@pytest.mark.parametrize("dim,heads,new", [(64, 2, 1), (128, 5, 4), (256, 2, 2)])
def test_rows_that_have_nothing_in_common_stand_alone(common, dim, heads, new):
    """A beam without continuations is emptied and grows anew among rows that go on from one prompt: these read it together
    all the same, as long as they are half of the group and two at least."""
    rng = np.random.default_rng(common + dim)
    cache, model, rows, _ = _branch(rng, 16, dim, 1, "e4m3", [6, 3], [common, 300], 40)
    whole = [common // 16 * 16 // 64 * 64] * 6 + [256] * 3

    def check(alone, kept):
        for r in alone:
            if model.lens[rows[r]] > 2:
                cache.free(_ids(rows[r]))
                model.free([rows[r]])
                _fill(cache, model, rng, [rows[r]], [1 + r % 2])
        counts = [int(min(c, model.lens[r])) for r, c in zip(rows, rng.integers(1, new + 1, 9))]
        counts[8] = new
        want = [0 if i in alone or not kept and i < 6 else n for i, n in enumerate(whole)]
        for kw in ({}, dict(window=90, sinks=3), dict(softcap=20.0)):
            _, b, _, _ = _check(cache, model, rng, rows, counts, [6, 3], heads, **kw)
            info = b._info[4:].view(-1, 8)[:, 2].tolist()
            assert info == [whole[0] if kept else 0, 256] + want
            assert b.shared.tolist() == [0] * 6 + whole[6:]
    check([3], True)
    check([1, 3, 5], True)
    check([1, 2, 3, 5], False)
    cache.reorder(_ids(*rows[:6]), _ids(0, 0, 4, 4, 4, 0))        # all live again, from two rows
    model.reorder(rows[:6], [0, 0, 4, 4, 4, 0])
    _, b, _, _ = _check(cache, model, rng, rows, [1] * 9, [6, 3], heads)
    assert b.shared.tolist() == whole and b._info[4:].view(-1, 8)[:, 2].tolist() == [whole[0], 256] + whole
    check([0], False)                                             # what others are compared with


def test_two_rows_of_which_one_stands_alone():
    rng = np.random.default_rng(1)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "int8", [1, 1, 1], [200, 100, 1], 0)
    for groups in ([2, 1], [1, 2], [3], [1, 1, 1]):
        _, b, _, _ = _check(cache, model, rng, rows, [1] * 3, groups, 2)
        alone = [192, 64, 0] if groups == [1, 1, 1] else [0, 0, 0] if groups[0] > 1 else [192, 0, 0]
        assert b.shared.tolist() == alone and b._info[4:].view(-1, 8)[len(groups):, 2].tolist() == alone


@pytest.mark.parametrize("heads", [2, 64])
def test_rows_with_more_tokens_than_max_new_are_left_as_they_were(heads):
    """For few and for many rows of queries; the others have their results."""
    rng = np.random.default_rng(heads)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [4], [200], 20)
    q = _bf16(rng, 10, heads, 64)
    b = kv.KvBatch(cache, _ids(*rows), _ids(1, 4, 2, 1), total=10, max_new=2)       # two tokens of no row
    assert int(cache.status.item()) == 4
    cache.status.zero_()
    out, lse = torch.full((10, heads, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((10, heads), 5.0, device="cuda")
    cache.attend_shared(0, q.cuda(), b, out=out, lse=lse)
    left = [1, 2, 3, 4, 8, 9]
    assert (out[left] == 3).all() and (lse[left] == 5).all()
    done = [0, 5, 6, 7]
    want, ref, slack, spread = model.attend(0, _f64(q)[done], [rows[0], rows[2], rows[3]], [0, 1, 3, 4])
    assert np.all(np.abs(_f64(out[done]) - want) <= S.attend_bound(want, slack, spread))
    assert np.all(np.abs(_f64(lse[done]) - ref) <= slack + 2.0 ** -20 * (1 + np.abs(ref)))


@pytest.mark.parametrize("dim,kv_heads,heads", [(64, 2, 2), (128, 1, 3)])
def test_many_groups(dim, kv_heads, heads):
    """More groups than a wave looks through at a time, some of them empty, of one row, or without common tokens."""
    rng = np.random.default_rng(dim)
    sizes = [int(x) for x in rng.integers(1, 4, 150)]
    cache, model, rows, _ = _branch(rng, 16, dim, kv_heads, "e4m3", sizes, [int(x) for x in rng.integers(1, 260, 150)], 20)
    n = sum(sizes)
    _check(cache, model, rng, rows, [1] * n, sizes, heads)
    groups = []
    for x in sizes:
        groups += [0] * int(rng.integers(0, 3)) + [x]
    _check(cache, model, rng, rows, [1] * n, groups + [0], heads, window=70)
    counts = [int(min(c, model.lens[r])) for r, c in zip(rows, rng.integers(0, 4, n))]
    _check(cache, model, rng, rows, counts, sizes, heads, softcap=20.0)


@pytest.mark.parametrize("dim,heads,rows,new", [(64, 63, 3, 1), (192, 31, 4, 2), (256, 9, 30, 7), (128, 21, 10, 3), (192, 1, 90, 1)])
def test_stacks_of_every_shape(dim, heads, rows, new):
    """Query heads that leave a row of tiles unfilled, just below what goes to the attention of many rows, and large stacks at
    the widths that take 16 rows at a time."""
    rng = np.random.default_rng(dim + heads)
    cache, model, order, _ = _branch(rng, 32, dim, 1, "int8", [rows], [500], 60)
    counts = [int(c) for c in rng.integers(0, new + 1, rows)]
    counts[rows // 2] = new
    for kw in ({}, dict(window=77, sinks=5)):
        _check(cache, model, rng, order, counts, [rows], heads, **kw)


def test_everything_first_called_in_a_capture():
    """Plan, attention, selection and move without a call before the capture: their workspaces are the graph's, and every
    replay has them as a first call does."""
    rng = np.random.default_rng(3)
    cache, model, rows, _ = _branch(rng, 16, 64, 1, "e4m3", [4], [300], 40)
    ids, q = _ids(*rows), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    x, scores, parents = torch.zeros(4, 9000, device="cuda"), torch.zeros(4, device="cuda"), _ids(0, 1, 2, 3)
    beams, graph, side = beam.Beams(1, 4), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            plan = kv.KvBatch(cache, ids)
            got, lse = cache.attend_shared(0, q, plan, lse=True)
            best = beams.select(x, scores)
            cache.reorder(ids, parents)
    torch.cuda.synchronize()
    for step in range(5):
        new = _bf16(rng, 4, 2, 64)
        y = torch.from_numpy(rng.standard_normal((4, 9000)).astype(np.float32))
        s = [-float(v) for v in rng.random(4)]
        moved = [int(p) for p in rng.integers(0, 4, 4)]
        q.copy_(new), x.copy_(y), scores.copy_(torch.tensor(s)), parents.copy_(_ids(*moved))
        graph.replay()
        torch.cuda.synchronize()
        out, ref, slack, spread = model.attend(0, _f64(new), rows)
        assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread)), step
        _choices(y, s, 4, 4, got=best)
        model.reorder(rows, moved)
        _same(cache, model, ("refs", "table", "lens"))
        _fill(cache, model, rng, rows, [1, 2, 17, 1])                # eager work between the replays
