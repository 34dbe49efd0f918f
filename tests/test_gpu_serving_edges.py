"""The serving operators on the GPU where they are used in less usual ways:
calls first made in a capture, cache entries that exist nowhere, values that
are not finite, soft caps of any size, long rows of every head size."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import kv
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf16(rng, *shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).bfloat16()


def _f64(t):
    return t.cpu().float().numpy().astype(np.float64)


def _filled(rng, lens, size=1.0, **kw):
    """A cache and its model, with rows of these lengths in layer 0."""
    kw = dict(dict(layers=1, max_seqs=len(lens), page_tokens=64, dtype="e4m3"), **kw)
    page = kw["page_tokens"]
    need = [-(-n // page) for n in lens]
    kw = dict(dict(n_pages=sum(need) + 2, max_pages=max(need) + 1), **kw)
    cache, model = kv.KvCache(**kw), S.Cache(**kw)
    rows, at = list(range(len(lens))), [0] + [int(x) for x in np.cumsum(lens)]
    k, v = (_bf16(rng, at[-1], kw["kv_heads"], kw["head_dim"], size=size) for _ in range(2))
    cache.extend(_ids(*rows), _ids(*lens))
    model.extend(rows, lens)
    cache.append(0, k.cuda(), v.cuda(), _ids(*rows), _ids(*at), max_new=max(lens))
    model.append(0, _f64(k), _f64(v), rows, at)
    torch.cuda.synchronize()
    return cache, model


def test_attention_first_called_in_a_capture():
    """Graphs captured with no workspace made before: an eager call and a later
    graph that come before the first one's replay are right, and so is every
    replay."""
    rng = np.random.default_rng(41)
    cache, _ = _filled(rng, [3000, 2000, 100, 7], kv_heads=1, head_dim=64)
    q, rows = _bf16(rng, 4, 16, 64).cuda(), _ids(0, 1, 2, 3)
    fresh = lambda: kv.KvCache.over(cache.k, cache.v, cache.scale, cache.refs, cache.table, cache.lens, 64)   # noqa: E731
    want = {n: cache.attend(0, q[:n], rows[:n], lse=True) for n in (1, 2, 4)}
    twin = fresh()
    full = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    del full                                         # memory that is not zero, for whoever asks next
    for n in (1, 2):
        out, lse = torch.zeros(n, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(2):
                twin.attend(0, q[:n], rows[:n], out=out, lse=lse)
        graphs.append(g), outs.append((out, lse))
    got = twin.attend(0, q, rows, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[4][0]) and torch.equal(got[1], want[4][1])
    for _ in range(3):
        for i in (1, 0):
            outs[i][0].zero_(), outs[i][1].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], want[i + 1][0]) and torch.equal(outs[i][1], want[i + 1][1])
        got = twin.attend(0, q, rows)
        torch.cuda.synchronize()
        assert torch.equal(got, want[4][0])


def test_growth_by_more_pages_than_32_bits_count():
    """1024 rows of 2^22 pages each: the pages wanted are 2^32, a sum that wraps
    to 0 would let the rows grow with no pages of their own."""
    n, pages = 1024, 1 << 22
    cache = kv.KvCache(1, 1, 1, 64, n, pages, page_tokens=16)
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    for last in (16 * pages, 16 * pages - 15, 1, 0):
        counts = torch.full((n,), 16 * pages, dtype=torch.int32, device="cuda")
        counts[-1] = last
        cache.extend(rows, counts)
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 1, last
        cache.status.zero_()
        assert not cache.lens.any() and not cache.refs.any()
    cache.extend(rows[:64], torch.ones(64, dtype=torch.int32, device="cuda"))
    cache.check()
    assert torch.equal(cache.table[:64, 0], rows[:64]) and bool((cache.refs == 1).all())
