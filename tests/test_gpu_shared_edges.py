"""Corners of the attention of groups, on the GPU."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from oracle import serving as S
from test_gpu_kv import _bf16, _f64, _fill, _ids
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
