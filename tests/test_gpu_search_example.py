"""The example that runs the plan, attention of groups, the choice of beams and
the move of rows together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


def _example():
    spec = importlib.util.spec_from_file_location("beam_search", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_search_stays_near_the_plain_layer():
    """Keys and values in int8 are off by 2.6% (rms) or less of a value: a step
    is at most amax / 64, errors are uniform, amax is at most 5 times the rms,
    and pages are rounded again when their scale grows.  Attention averages the
    values and moves logits by as much, so its result is off by less than twice
    that; the residual beside it is rounded to BF16 (2^-9 rms at most), and the
    output projection keeps relative distances."""
    words, worst = _example().run(steps=6, log=lambda s: print(s, flush=True))
    assert worst < 0.052 + 2 ** -8
    assert len(words) == 8 and all(len(w) == 6 and min(w) >= 0 for w in words)


def test_one_beam_of_each_request():
    """Groups of a single row, whose own tokens are all that it has in common."""
    words, worst = _example().run(steps=4, requests=3, beams=1, prompt=70, seed=1, log=lambda s: print(s, flush=True))
    assert worst < 0.052 + 2 ** -8 and all(len(w) == 4 for w in words)
