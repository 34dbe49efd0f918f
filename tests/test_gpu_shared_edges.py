"""Corners of the attention of groups, on the GPU."""
import numpy as np
import pytest

from test_gpu_shared import _branch, _check

pytestmark = pytest.mark.gpu

@pytest.mark.parametrize("dim,heads,own", [(64, 2, 200), (256, 3, 90), (128, 4, 3000)])
def test_rows_of_no_groups(dim, heads, own):
    """Offsets of no groups: every row by itself, whole and split."""
    rng = np.random.default_rng(dim)
    cache, model, rows, _ = _branch(rng, 16, dim, 1, "int8", [3, 1, 5], [100, 70, 300], own)
    _check(cache, model, rng, rows, [1] * 9, [], heads)
    _check(cache, model, rng, rows, [1, 0, 2, 1, 3, 1, 1, 0, 2], [], heads, window=50, sinks=2)
