"""Rows of logits at the ends of their type, and equal scores, on the GPU."""
import math

import pytest
import torch

from lossless_entropy_coding_amd import beam
from test_gpu_beam import INF, _check, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab", [300, 40000])
def test_rows_of_large_logits_keep_their_scores(half, vocab):
    """Rows whose mask, the type's lowest value, leaves nothing are uniform over all tokens, and those that are large
    everywhere are as the same ones near 0: a score is not lost beside its logits."""
    dt = torch.bfloat16 if half else torch.float32
    x, s = _logits(vocab, 6, vocab, half)
    x[0] = torch.finfo(dt).min
    x[1, ::7] = torch.finfo(dt).min
    x[2] = torch.finfo(dt).max
    x[3] = 1e12
    x[4] = -1e20
    x[4, :3] = 1e30
    for beams, keep in ((1, 2), (2, 5), (6, 7)):
        _check(x, s, beams, keep)
        _check(x, s, beams, keep, softcap=30.0)
    got = beam.Beams(6, 1, keep=1).select(x.cuda(), torch.tensor(s).cuda())
    # the sum is right to 2^-17, and a score of up to 32 is rounded to 2^-20
    for row, tokens in ((0, vocab), (2, vocab), (3, vocab), (4, 3)):
        assert abs(float(got.scores[row, 0]) - (s[row] - math.log(tokens))) <= 2.0 ** -17 + 2.0 ** -20
    got = beam.Beams(6, 1, keep=1).select(x.cuda(), torch.tensor(s).cuda(), softcap=1e30)
    assert abs(float(got.scores[0, 0]) - (s[0] - math.log(vocab))) <= 2.0 ** -17 + 2.0 ** -20


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("softcap", [0.5, 30.0, 300.0])
@pytest.mark.parametrize("keep", [1, 2, 5, 40])
def test_saturated_logits_keep_their_order(half, softcap, keep):
    """Where tanh is 1 in 64 bits scores are equal, and a beam's tokens still go by their logits, beams by their number."""
    dt = torch.bfloat16 if half else torch.float32
    x = torch.zeros(4, 3000)
    for row in range(4):
        x[row, torch.arange(50) * 53 + row] = softcap * (32 + torch.arange(50).roll(11 * row))     # all apart in 8 bits
    x[1] = x[0]
    x = x.to(dt)
    got = beam.Beams(2, 2, keep=keep).select(x.cuda(), torch.zeros(4, device="cuda"), softcap=softcap)
    best = x[0].float().argsort(descending=True, stable=True)[:keep].tolist()
    assert got.scores[0].unique().numel() == 1
    assert got.parents[0].tolist() == [0] * keep and got.tokens[0].tolist() == best
    _check(x, [0.0, 0.0, -1.0, -2.0], 2, keep, softcap=softcap)


def test_the_most_beams_of_a_call():
    """65535 of them, one to a request and 64; a few requests are looked at."""
    for batch, beams, vocab in ((65535, 1, 19), (1023, 64, 130)):
        x, s = _logits(batch, batch * beams, vocab, True)
        got = beam.Beams(batch, beams, keep=3).select(x.cuda(), torch.tensor(s).cuda())
        for at in (0, 1, batch // 2, batch - 1):
            part = type(got)(*(t[at:at + 1] for t in got))
            part = part._replace(parents=part.parents - at * beams)
            rows = slice(at * beams, (at + 1) * beams)
            _check(x[rows], s[rows], beams, 3, got=part)


@pytest.mark.parametrize("half", [True, False])
def test_rows_more_than_4_gib_apart(half):
    x, s = _logits(3, 4, 5001, half)
    stride = (1 << 31) + 7 if half else (1 << 30) + 5
    flat = torch.empty(3 * stride + 5001, dtype=x.dtype, device="cuda")
    rows = flat.as_strided((4, 5001), (stride, 1))
    rows.copy_(x)
    _check(x, s, 2, 4, got=beam.Beams(2, 2, keep=4).select(rows, torch.tensor(s).cuda()))
