"""The example that runs adapters, cache, attention and page upkeep together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")


def test_a_served_layer_stays_near_the_plain_one():
    """Keys and values in int8 with a power-of-two scale per page: a step is at
    most amax / 64 and errors are uniform, so a value is off by amax / 64 /
    sqrt(12) (rms), times sqrt(4/3) for the roundings when a page's scale
    grows.  With amax of at most 5 times the rms of a page's values that is
    2.6% of a value; the attention averages values (the error with them) and
    logits of size ~1 move by 2.6% of one channel's share, so the layer's
    result is off by less than twice that."""
    spec = importlib.util.spec_from_file_location("serve_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.run(steps=4, log=lambda s: print(s, flush=True)) < 0.052
