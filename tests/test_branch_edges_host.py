"""Corners of the operators for several continuations that need no GPU: buffers
that lie over each other, workspaces, the references at the ends of a type."""
import math

import numpy as np
import pytest

from oracle import serving as S


# --------------------------------------------------------------------- beams
@pytest.mark.parametrize("value", [-3.4e38, 3.4e38, 1e12, 0.0])
def test_the_reference_keeps_scores_beside_large_logits(value):
    """A row of one value is uniform over its tokens, whatever the value is."""
    x = np.full((2, 50), value)
    x[1] = np.linspace(-1, 1, 50)
    out, tok, par, _, _, _ = S.select(x, np.array([-5.0, -40.0]), 2, 3)
    np.testing.assert_allclose(out, [[-5.0 - math.log(50)] * 3], rtol=1e-12)
    assert tok.tolist() == [[0, 1, 2]] and par.tolist() == [[0, 0, 0]]
