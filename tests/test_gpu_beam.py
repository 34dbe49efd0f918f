"""The choice of continuations on the GPU against its 64-bit form
(oracle.serving.select): tokens, parents and ends equal, scores within the bound
that is derived there."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import beam
from oracle import serving as S

pytestmark = pytest.mark.gpu
INF = float("inf")


def _check(logits, scores, beams, keep, done=None, eos=-1, softcap=0.0, got=None):
    """logits: a CPU tensor of the type that is sent, or (with got) the values."""
    if got is None:
        b = beam.Beams(logits.shape[0] // beams, beams, keep=keep, eos=eos)
        got = b.select(logits.cuda(), torch.tensor(scores, dtype=torch.float32).cuda(),
                       done=None if done is None else torch.tensor(done, dtype=torch.int32).cuda(), softcap=softcap)
    scores = np.float32(scores).astype(np.float64).reshape(-1)
    s, t, p, d, gaps, loose = S.select(logits.float().numpy().astype(np.float64), scores, beams, keep, done, eos, softcap)
    real = np.isfinite(s)
    bound = loose[:, None] + 2.0 ** -24 * np.abs(np.where(real, s, 0)) + 1e-300
    # what is next to a border would be decided by rounding: such inputs say nothing
    assert ((gaps == 0) | (gaps > 2 * bound)).all(), "near ties: another seed"
    for a, b in ((got.tokens, t), (got.parents, p), (got.done, d)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    g = got.scores.cpu().numpy().astype(np.float64)
    assert (np.isneginf(g) == ~real).all()
    off = np.abs(np.where(real, g, 0) - np.where(real, s, 0))
    assert (off <= bound).all(), off.max() / bound.max()


def _logits(seed, rows, vocab, half, size=3.0):
    g = torch.Generator().manual_seed(seed)
    x = size * torch.randn(rows, vocab, generator=g)
    # values all over their type's steps, so that ties within a row are ties and others are far apart
    return (x.bfloat16() if half else x), (-9 * torch.rand(rows, generator=g)).tolist()


@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 1000, 4095, 4097, 32771, 50257])
@pytest.mark.parametrize("half", [True, False])
def test_sizes_of_the_vocabulary(vocab, half):
    for batch, beams, keep, seed in ((1, 1, 1, 0), (2, 4, 4, 1), (3, 3, 6, 2)):
        x, s = _logits(seed + vocab, batch * beams, vocab, half)
        _check(x, s, beams, keep)


@pytest.mark.parametrize("beams,keep", [(1, 128), (5, 17), (16, 16), (64, 64), (64, 128), (2, 1)])
@pytest.mark.parametrize("half", [True, False])
def test_numbers_of_beams_and_of_the_kept(beams, keep, half):
    x, s = _logits(7 * beams + keep, 2 * beams, 3001, half)
    _check(x, s, beams, keep)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("batch,beams,vocab", [(1, 2, 256000), (40, 4, 70001), (300, 2, 20000)])
def test_parts_of_every_size(half, batch, beams, vocab):
    """From one vector a thread to eight."""
    x, s = _logits(vocab, batch * beams, vocab, half)
    _check(x, s, beams, 4)


@pytest.mark.parametrize("softcap", [0.5, 30.0, 256.0, 1000.0, 1e30, INF])
def test_soft_caps(softcap):
    x, s = _logits(11, 6, 5003, False, size=4.0)
    b = beam.Beams(2, 3, keep=5)
    got = b.select(x.cuda(), torch.tensor(s).cuda(), softcap=softcap)
    _check(x, s, 3, 5, softcap=0.0 if softcap > 1e9 else softcap, got=got)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("offset,stride", [(0, 1009), (1, 1009), (3, 1016), (5, 2000), (8, 1003)])
def test_rows_at_any_address(half, offset, stride):
    """Rows that begin anywhere between two 16-B boundaries, with other values before, between and after them."""
    x, s = _logits(offset + stride, 8, 1001, half)
    flat = torch.full((offset + 8 * stride + 9,), 1000.0, dtype=x.dtype, device="cuda")
    rows = flat[offset:offset + 8 * stride].view(8, stride)[:, :1001]
    rows.copy_(x)
    assert rows.data_ptr() % 16 == flat[offset:].data_ptr() % 16
    got = beam.Beams(2, 4, keep=6).select(rows, torch.tensor(s).cuda())
    _check(x, s, 4, 6, got=got)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("keep", [3, 16, 40, 128])
def test_ties_go_to_the_lowest_token_and_beam(half, keep):
    """Rows of one value, of two, and of few: far more equal logits than a list holds; beams that are equal."""
    dt = torch.bfloat16 if half else torch.float32
    g = torch.Generator().manual_seed(keep)
    for vocab in (40, 9000, 33000):
        rows = [torch.full((vocab,), 1.5), torch.randint(0, 2, (vocab,), generator=g).float(), torch.randint(0, 6, (vocab,), generator=g).float(),
                -torch.zeros(vocab)]
        x = torch.stack([r for r in rows for _ in range(2)]).to(dt)
        _check(x, [-1.0] * 8, 2, keep)


@pytest.mark.parametrize("half", [True, False])
def test_the_largest_logits_of_one_thread(half):
    """The largest logits are those that one group of threads reads, up to all of a thread's."""
    vec = 8 if half else 4
    x, s = _logits(5, 300 * 2, 40000, half)
    own = (torch.arange(40000) // vec) % 512
    for i, (lo, hi) in enumerate([(3, 4), (64, 66), (7, 8)]):
        x[2 * i, (own >= lo) & (own < hi)] += 50.0
        x[2 * i + 1, own % 64 == 5] += 50.0
    for keep in (16, 17, 128):
        b = beam.Beams(300, 2, keep=keep)
        got = b.select(x.cuda(), torch.tensor(s).cuda())
        first = type(got)(*(t[:3] for t in got))
        _check(x[:6], s[:6], 2, keep, got=first)


def test_masks_dead_beams_and_what_is_no_number():
    x, s = _logits(21, 12, 2500, False)
    x[0, 3:] = -INF                                  # three tokens are allowed
    x[1] = -INF                                      # none is
    x[2, 77] = float("nan")
    x[3, 78] = INF
    x[4] = float("nan")
    x[5, :2499] = -INF
    x[6, ::2] = -3e38
    x[7] = -3e38
    s[8], s[9], s[10] = -INF, float("nan"), INF
    for beams, keep in ((3, 5), (1, 4), (12, 12), (6, 128)):
        _check(x, s, beams, keep)
        _check(x, s, beams, keep, softcap=30.0)
    _check(torch.full((4, 300), -INF), [0.0] * 4, 2, 3)


def test_ends_of_beams():
    x, s = _logits(33, 8, 900, True)
    x[:, 2] = 14.0                                   # the end is likely, and as likely everywhere
    done = [0, 1, 0, 0, 1, 1, 1, 1]
    x[5] = float("nan")                              # not read
    s[6] = -INF
    _check(x, s, 4, 6, done=done, eos=2)
    _check(x, s, 2, 3, done=done, eos=2)
    _check(x[:1], s[:1], 1, 3, eos=2)
    _check(x, s, 4, 6, done=[-1] * 8, eos=899)


def test_the_first_step_has_one_beam():
    x, _ = _logits(2, 4, 10000, True)
    x[:] = x[0]
    _check(x, [0.0, -INF, -INF, -INF], 4, 4)


def test_streams_captures_and_more_calls_of_one_handle():
    """A captured choice replays on new logits; eager calls of other sizes go on in between; the results of earlier
    calls stay."""
    b = beam.Beams(2, 4, keep=4, eos=1)
    x, s = _logits(1, 8, 7001, True)
    dev, sc, done = x.cuda(), torch.tensor(s).cuda(), torch.zeros(8, dtype=torch.int32, device="cuda")
    b.select(dev, sc, done=done)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = b.select(dev, sc, done=done)
    torch.cuda.current_stream().wait_stream(side)
    eager = []
    for i in range(4):
        x, s = _logits(50 + i, 8, 7001, True)
        dev.copy_(x)
        sc.copy_(torch.tensor(s))
        graph.replay()
        torch.cuda.synchronize()
        _check(x, s, 4, 4, eos=1, got=kept)
        y, r = _logits(80 + i, 8, 200 + 40000 * i, False)       # the workspace grows
        eager.append((y, r, b.select(y.cuda(), torch.tensor(r).cuda())))
    for y, r, got in eager:
        _check(y, r, 4, 4, eos=1, got=got)


def test_empty_batches():
    got = beam.Beams(0, 4).select(torch.zeros(0, 10, device="cuda"), torch.zeros(0, device="cuda"))
    assert got.scores.shape == (0, 4)


@pytest.mark.parametrize("half,vocab", [(True, 1000000), (False, 1000000), (False, 524285), (True, 262145)])
def test_the_largest_vocabularies(half, vocab):
    """Up to 64 parts of a row, of the largest size."""
    x, s = _logits(vocab, 4, vocab, half)
    x[:, -1] += 9.0
    x[:, 0] += 8.0
    _check(x, s, 4, 5)
    flat = torch.empty(4 * vocab + 3, dtype=x.dtype, device="cuda")
    rows = flat[3:].view(4, vocab)
    rows.copy_(x)
    _check(x, s, 4, 5, got=beam.Beams(1, 4, keep=5).select(rows, torch.tensor(s).cuda()))
