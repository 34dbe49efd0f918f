"""Corners of the plan of a step's tokens and of the moves of rows, on the GPU."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from test_gpu_branches import _branched, _plan_same
from test_gpu_kv import _ids, _pair, _same

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------- plans
@pytest.mark.parametrize("common", [100, 30000])
def test_tokens_without_a_place_have_no_slot(common):
    """A row with more new tokens than max_new: flagged, its tokens have neither; the others keep theirs."""
    _, cache, model, order = _branched(3, 16, 1, 6, common, 10)
    b = kv.KvBatch(cache, _ids(*order), _ids(1, 5, 2, 1, 1, 1), total=11, max_new=2)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 4
    cache.status.zero_()
    want = model.batch(order, [1, 5, 2, 1, 1, 1], [0, 6], 11, cache.max_pages)
    want[1][1:6] = want[2][1:6] = -1
    _plan_same(b, want)


def test_a_plan_of_its_own_rows():
    """The one buffer of a plan that may be given back to it."""
    _, cache, model, order = _branched(4, 16, 2, 3, 200, 30)
    b = kv.KvBatch(cache, _ids(*order), groups=_ids(0, 3, 6))
    b.update(b.rows, groups=_ids(0, 3, 6))
    _plan_same(b, model.batch(order, [1] * 6, [0, 3, 6], 6, cache.max_pages))
    for own in (b.lead, b.shared, b.places, b.starts[:6]):
        with pytest.raises(Exception, match="overlaps"):
            b.update(own, groups=_ids(0, 3, 6))
    cache.check()


def test_plans_of_rows_far_longer_than_said():
    """width and max_len decide the size of the table and no more: rows of 2^27 tokens, named 512 times in all, whose pages differ from
    the first one on."""
    t = lambda *s, k=torch.int32: torch.zeros(*s, dtype=k, device="cuda")     # noqa: E731
    table = t(2, 1 << 23)
    table[1] = 1
    cache = kv.KvCache.over(t(1, 2, 1, 16, 64, k=torch.uint8), t(1, 2, 1, 64, 16, k=torch.uint8), t(1, 2, 1, 2, k=torch.float32),
                            t(2), table, t(2).fill_(1 << 27), head_dim=8)
    b = kv.KvBatch(cache, _ids(*[0, 1] * 256), max_len=16)
    assert int(b.shared.abs().max()) == 0 and b.places.unique().tolist() == [(1 << 27) - 1] and b.table.flatten().tolist() == [0, 1] * 256
    b.update(_ids(*[1] * 512))
    assert b.shared.unique().tolist() == [1 << 27]
    cache.check()


@pytest.mark.parametrize("times", [1, 100])
@pytest.mark.parametrize("common", [100, 30000])
def test_groups_that_do_not_hold(common, times):
    """In plans of every size, rows named once or many times: flagged, nothing in common (a token counted twice would be seen
    twice), attention still right, and the next plan is whole again."""
    _, cache, model, order = _branched(8, 16, 1, 6, common, 10)
    rng = np.random.default_rng(0)
    cache.k.random_(0, 60)
    cache.v.random_(0, 60)
    cache.scale.fill_(2.0 ** -5)
    rows, n = order * times, 6 * times
    q = torch.from_numpy(rng.standard_normal((n, 2, 8)).astype(np.float32)).bfloat16().cuda()
    want = cache.attend(0, q, _ids(*rows))
    whole = model.batch(rows, [1] * n, [0, n], n, cache.max_pages)
    for offs in ([0, 4 * times, 2 * times, n], [0, 5, 3, n], [-5, 2, n], [0, n + 1], [0, 1 << 30], [n, 0], [3, -(1 << 31), n], [1, n, 2]):
        b = kv.KvBatch(cache, _ids(*rows), groups=_ids(*offs))
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 4, offs
        cache.status.zero_()
        assert int(b.shared.abs().max()) == 0 and int(b._info[4:].view(-1, 8)[:, 2].abs().max()) == 0, offs
        _plan_same(b, (*whole[:4], b.lead.cpu().numpy(), np.zeros(n, np.int32)))
        assert int(b.lead.min()) >= 0 and (b.lead.cpu().numpy() <= np.arange(n)).all()
        got = cache.attend_shared(0, q, b)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max(), offs
        good = sorted([0, n] + [int(x) for x in rng.integers(0, n + 1, len(offs) - 2)])
        b.update(_ids(*rows), groups=_ids(*good))
        _plan_same(b, model.batch(rows, [1] * n, good, n, cache.max_pages))
        got = cache.attend_shared(0, q, b)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max(), good
    cache.check()


@pytest.mark.parametrize("times", [1, 100])
@pytest.mark.parametrize("common", [100, 30000])
def test_rows_and_counts_that_do_not_hold(common, times):
    """In plans of every size: flagged, unknown rows have no place and nothing in common, the others keep what is theirs."""
    _, cache, model, order = _branched(9, 16, 1, 6, common, 10)
    rows, n = order * times, 6 * times
    counts = [1] * n
    most = cache.max_pages

    def flagged(rows, counts, total):
        b = kv.KvBatch(cache, _ids(*rows), _ids(*counts), total=total)
        first = [t.clone() for t in (b.starts, b.places, b.slots, b.table, b.lead, b.shared, b._info)]
        b.update(_ids(*rows), _ids(*counts))                        # the same again: nothing is left over
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 4 and int(b._info[0]) == 0
        assert all(torch.equal(x, y) for x, y in zip(first, (b.starts, b.places, b.slots, b.table, b.lead, b.shared, b._info)))
        cache.status.zero_()
        return b
    for bad in (7, -1, 1 << 30, -(1 << 31)):                        # rows 0..6 exist
        b = flagged([rows[0], bad] + rows[2:], counts, n)
        assert int(b.places[1]) == int(b.slots[1]) == -1 and (b.table[1] == -1).all() and int(b.shared.max()) == 0
        want = model.batch(rows, counts, [0, n], n, most)
        assert b.places[2:].tolist() == want[1][2:].tolist() and b.slots[2:].tolist() == want[2][2:].tolist()
        b = flagged([bad] + rows[1:], counts, n)                    # the group's first
        assert int(b.shared.max()) == 0 and int(b._info[4:].view(-1, 8)[:, 2].max()) == 0
    b = flagged(rows, [1, -3, 2] + counts[3:], n)
    assert b.starts[:4].tolist() == [0, 1, 1, 3]
    b = flagged(rows, [1] * (n - 1) + [1 << 30], n)
    assert b.starts[-2:].tolist() == [n - 1, n]
    b = flagged(rows, counts, n + 2)
    assert b.places[n:].tolist() == [-1, -1] and b.slots[n:].tolist() == [-1, -1]
    b = flagged(rows, [2] * n, 2 * n - 1)
    assert int(b.starts[n]) == 2 * n - 1
    b = kv.KvBatch(cache, _ids(*rows))
    _plan_same(b, model.batch(rows, counts, [0, n], n, most))
    cache.check()


# ------------------------------------------------------------------- reorder
def test_moves_of_rows_of_many_pages():
    """More blocks of columns than a launch has workgroups for: each takes several."""
    rng = np.random.default_rng(5)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=8, n_pages=3000, max_seqs=520, max_pages=66000, page_tokens=16, dtype="int8")
    rows = [int(r) for r in rng.permutation(520)]
    model.lens[rows] = [65990 * 16 - 3, 65537 * 16] + [int(c) for c in rng.integers(0, 40, 518)]
    for r in rows:                                               # pages of any row, the last thousand are free
        held = model.table[r, :model.pages(model.lens[r])]
        held[:] = rng.integers(0, 2000, len(held))
        np.add.at(model.refs, held, 1)
    for name in ("table", "lens", "refs"):
        getattr(cache, name).copy_(torch.from_numpy(getattr(model, name)))
    for step in range(3):
        parents = [int(q) for q in rng.permutation(520)]
        parents[7], parents[8] = parents[int(rng.integers(0, 7))], -1
        cache.reorder(_ids(*rows), _ids(*parents))
        model.reorder(rows, parents)
        _same(cache, model)
        assert model.status == 0 and int(model.lens.max()) > 65536 * 16


def test_moves_in_the_widest_table_are_checked():
    """As many columns as a table can have, for as many rows as a call takes (named more than once, so nothing moves)."""
    t = lambda *s, k=torch.int32: torch.zeros(*s, dtype=k, device="cuda")     # noqa: E731
    cache = kv.KvCache.over(t(1, 4, 1, 16, 64, k=torch.uint8), t(1, 4, 1, 64, 16, k=torch.uint8), t(1, 4, 1, 2, k=torch.float32),
                            t(4), t(1, (1 << 27) - 16), t(1).fill_(40), head_dim=8)
    for n in (129, 4096):
        cache.reorder(t(n), t(n))
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 4 and cache.lens.tolist() == [40]
        cache.status.zero_()
    cache.reorder(t(1), t(1).fill_(-1))
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [0]
