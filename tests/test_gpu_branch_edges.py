"""Corners of the plan of a step's tokens and of the moves of rows, on the GPU."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from test_gpu_branches import _branched, _plan_same
from test_gpu_kv import _ids

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
