"""The paged 8-bit key/value cache on the GPU against its plain model
(oracle.serving.Cache): pages, stored codes and scales equal bit for bit;
attention within the bound that attend_bound derives."""
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


def _pair(**kw):
    """A cache with stale bytes everywhere (past head_dim the keys are zero), and its model."""
    cache, model = kv.KvCache(**kw), S.Cache(**kw)
    rng = np.random.default_rng(99)
    model.k[..., :kw["head_dim"]] = rng.integers(0, 256, model.k[..., :kw["head_dim"]].shape)
    model.v[:] = rng.integers(0, 256, model.v.shape)
    model.scale[:] = np.nan
    for name in ("k", "v", "scale"):
        getattr(cache, name).copy_(torch.from_numpy(getattr(model, name)))
    return cache, model


def _same(cache, model, names=("refs", "table", "lens", "k", "v", "scale")):
    torch.cuda.synchronize()
    for n in names:
        a, b = getattr(cache, n).cpu().numpy(), getattr(model, n)
        assert a.tobytes() == np.ascontiguousarray(b).tobytes(), n
    assert int(cache.status.item()) == model.status


def _fill(cache, model, rng, rows, counts, sizes=(1.0,), f32=False, layers=None):
    """extend, then append to every layer, on both sides."""
    cache.extend(_ids(*rows), _ids(*counts))
    model.extend(rows, counts)
    starts = [0] + [int(x) for x in np.cumsum(counts)]
    for layer in range(cache.layers) if layers is None else layers:
        size = sizes[layer % len(sizes)]
        k, v = (_bf16(rng, starts[-1], cache.kv_heads, cache.head_dim, size=size) for _ in range(2))
        if f32:
            k, v = k.float() * 1.001, v.float() * 0.999
        cache.append(layer, k.cuda(), v.cuda(), _ids(*rows), _ids(*starts), max_new=max(counts))
        model.append(layer, _f64(k), _f64(v), rows, starts)


# --------------------------------------------------------------------- pages
@pytest.mark.parametrize("seed,page", [(0, 16), (1, 32), (2, 16), (3, 64)])
def test_pages_follow_the_model(seed, page):
    """Random growth, forks, frees and compactions of a small pool, some of
    them refused for want of pages or room; every buffer after every call."""
    rng = np.random.default_rng(seed)
    cache, model = _pair(layers=2, kv_heads=1, head_dim=24, n_pages=40, max_seqs=10, max_pages=9, page_tokens=page, dtype="int8")
    # scales: the model's NaN bits are compared as they are
    for step in range(40):
        used = [r for r in range(10) if model.lens[r]]
        empty = [r for r in range(10) if not model.lens[r]]
        op = rng.choice(["extend", "extend", "fork", "free", "compact"])
        print("step", step, op, flush=True)
        if op == "extend":
            rows = [int(r) for r in rng.permutation(10)[:rng.integers(1, 6)]]
            counts = [int(c) for c in rng.integers(0, 3 * page, len(rows))]
            cache.extend(_ids(*rows), _ids(*counts))
            model.extend(rows, counts)
        elif op == "fork" and used and empty:
            kids = empty[:rng.integers(1, len(empty) + 1)]
            parents = [int(rng.choice(used)) for _ in kids]
            cache.fork(_ids(*parents), _ids(*kids))
            model.fork(parents, kids)
        elif op == "free" and used:
            rows = used[:rng.integers(1, len(used) + 1)]
            cache.free(_ids(*rows))
            model.free(rows)
        elif op == "compact":
            cache.compact()
            model.compact()
        _same(cache, model)


def test_refused_page_calls_change_nothing():
    cache, model = _pair(layers=1, kv_heads=1, head_dim=16, n_pages=6, max_seqs=4, max_pages=4, page_tokens=16, dtype="e4m3")
    cache.extend(_ids(0, 1), _ids(40, 16))
    model.extend([0, 1], [40, 16])
    _same(cache, model)

    def refused(bit, call, *args):
        call(*args)
        model.status |= bit
        _same(cache, model)
        cache.status.zero_()
        model.status = 0
    refused(1, cache.extend, _ids(2, 1), _ids(40, 16))               # four pages wanted, two free
    refused(2, cache.extend, _ids(2, 0), _ids(1, 25))                # row 0 would be longer than its table row
    refused(4, cache.extend, _ids(2, 4), _ids(1, 1))                 # no row 4
    refused(4, cache.extend, _ids(2, -1), _ids(1, 1))
    refused(4, cache.extend, _ids(2), _ids(-1))
    refused(8, cache.fork, _ids(0), _ids(1))                         # the child is in use
    refused(4, cache.fork, _ids(0), _ids(0))
    refused(4, cache.fork, _ids(9), _ids(2))
    refused(4, cache.free, _ids(7))
    cache.extend(_ids(2), _ids(30))
    model.extend([2], [30])
    refused(1, cache.fork, _ids(0), _ids(3))                         # no page for the copy of the last one
    cache.free(_ids(1, 1))                                           # named twice: freed once
    model.free([1])
    _same(cache, model)
    with pytest.raises(RuntimeError, match="free pages"):
        cache.extend(_ids(3), _ids(60))
        cache.check()
    cache.check()
    # a count that is wrong already is reported and stays at 0
    cache.refs[cache.table[0, 0]] = 0
    cache.free(_ids(0))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 32 and int(cache.refs.min()) == 0


def test_bad_table_entries_are_reported_not_followed():
    cache, model = _pair(layers=1, kv_heads=2, head_dim=64, n_pages=8, max_seqs=3, max_pages=4, page_tokens=16, dtype="e4m3")
    rng = np.random.default_rng(1)
    _fill(cache, model, rng, [0, 1], [40, 20])
    q = _bf16(rng, 2, 2, 64).cuda()
    want = cache.attend(0, q, _ids(0, 1))
    cache.check()
    cache.table[0, 1] = 1 << 30
    got = cache.attend(0, q, _ids(0, 1))
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()
    assert torch.isfinite(got.float()).all() and torch.equal(got[1], want[1])
    before = cache.k.clone()
    cache.append(0, q, q, _ids(0, 1))                                # both rows' last tokens lie on good pages
    cache.check()
    cache.table[0, 2] = -5
    cache.append(0, q, q, _ids(0, 1))
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()
    assert before.shape == cache.k.shape
    cache.fork(_ids(0), _ids(2))
    cache.free(_ids(0))
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()
    out = cache.attend(0, q[:1], _ids(77))
    assert float(out.float().abs().max()) == 0
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()


def test_copy_pages_and_large_pool():
    """Copies in every layer; allocation, compaction over more than one block of counts."""
    rng = np.random.default_rng(4)
    cache, model = _pair(layers=3, kv_heads=2, head_dim=65, n_pages=9000, max_seqs=5, max_pages=4000, page_tokens=16, dtype="int8")
    src, dst = _ids(5, 8999, 4096), _ids(6, 0, 4097)
    cache.copy_pages(src, dst)
    for a, b in zip(src.tolist(), dst.tolist()):
        for n in ("k", "v", "scale"):
            getattr(model, n)[:, b] = getattr(model, n)[:, a]
    _same(cache, model)
    rows, counts = [0, 1, 2, 3], [16 * 3000, 16 * 2500 + 3, 0, 16 * 3400 - 1]
    cache.extend(_ids(*rows), _ids(*counts))
    model.extend(rows, counts)
    _same(cache, model, ("refs", "table", "lens"))
    cache.fork(_ids(1, 3), _ids(2, 4))
    model.fork([1, 3], [2, 4])
    cache.free(_ids(0, 1))
    model.free([0, 1])
    _same(cache, model)
    cache.compact()
    model.compact()
    _same(cache, model)
    cache.copy_pages(_ids(1, 9000), _ids(-1, 2))
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 2), (128, 64, 1), (80, 32, 3), (1, 16, 1), (256, 128, 1), (65, 256, 2)])
@pytest.mark.parametrize("f32", [False, True])
def test_append_stores_the_rule(dtype, dim, page, heads, f32):
    """Prompts, single tokens, growth of a page's scale by larger later tokens, tokens far below 2^-60, zeros."""
    print("append", dtype, dim, page, heads, f32, flush=True)
    rng = np.random.default_rng(dim + page)
    cache, model = _pair(layers=2, kv_heads=heads, head_dim=dim, n_pages=40, max_seqs=4, max_pages=8, page_tokens=page, dtype=dtype)
    rows = [2, 0, 3]
    _fill(cache, model, rng, rows, [page - 1, 3 * page + 5, 1], (1.0, 1e-3), f32)
    _same(cache, model)
    for size in (0.01, 4.0, 1e4, 0.0, 1e-25, 1e30):
        _fill(cache, model, rng, rows, [1, 1, 1], (size, 1.0 / (size + 1e-9)), f32)
        _same(cache, model)
    _fill(cache, model, rng, [0, 3], [0, 2 * page], (1.0,), f32)
    _same(cache, model)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page", [(64, 256), (96, 64), (128, 64), (256, 64), (256, 128), (8, 16)])
@pytest.mark.parametrize("f32", [False, True])
def test_append_of_chunks_anywhere_in_a_page(dtype, dim, page, f32):
    print("append chunks", dtype, dim, page, f32, flush=True)
    rng = np.random.default_rng(dim * page)
    cache, model = _pair(layers=1, kv_heads=2, head_dim=dim, n_pages=30, max_seqs=3, max_pages=10, page_tokens=page, dtype=dtype)
    for counts in ([1, 2, 3], [3, 5, 7], [4, 16, 17], [9, 30, 33], [page, page - 1, page + 1], [1, 4, 2 * page], [31, 2, 6]):
        _fill(cache, model, rng, [2, 0, 1], counts, (1.0, 0.01, 20.0), f32)
        _same(cache, model)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_append_of_non_finite_values(dtype):
    cache, model = _pair(layers=1, kv_heads=2, head_dim=64, n_pages=4, max_seqs=1, max_pages=4, page_tokens=16, dtype=dtype)
    rng = np.random.default_rng(3)
    cache.extend(_ids(0), _ids(20))
    model.extend([0], [20])
    k, v = _bf16(rng, 20, 2, 64), _bf16(rng, 20, 2, 64)
    k[3, 0, 5], k[4, 1, 6], v[17, 0, 7], v[18, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    cache.append(0, k.cuda(), v.cuda(), _ids(0), _ids(0, 20))
    with np.errstate(invalid="ignore"):
        model.append(0, _f64(k), _f64(v), [0], [0, 20])
    _same(cache, model)
    with pytest.raises(RuntimeError, match="non-finite"):
        cache.check()


def test_append_reads_strided_tokens_and_refuses_bad_ranges():
    rng = np.random.default_rng(8)
    cache, model = _pair(layers=1, kv_heads=2, head_dim=64, n_pages=8, max_seqs=3, max_pages=4, page_tokens=16, dtype="e4m3")
    qkv = _bf16(rng, 30, 7, 64)                                      # queries, keys and values of one projection
    cache.extend(_ids(1, 2), _ids(20, 10))
    model.extend([1, 2], [20, 10])
    d = qkv.cuda()
    cache.append(0, d[:, 3:5], d[:, 5:7], _ids(1, 2), _ids(0, 20, 30))
    model.append(0, _f64(qkv)[:, 3:5], _f64(qkv)[:, 5:7], [1, 2], [0, 20, 30])
    _same(cache, model)
    odd = torch.zeros(30 * 7 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    odd[1:] = d.reshape(-1)
    u = odd[1:].view(30, 7, 64)                                      # 2 bytes past 16-B alignment
    cache.append(0, u[:, 3:5], u[:, 5:7], _ids(1, 2), _ids(0, 20, 30))
    _same(cache, model)
    before = cache.k.clone(), cache.v.clone(), cache.scale.clone()
    for starts in ((0, 21, 30), (0, 20, 31), (5, 0, 30), (-1, 19, 29)):
        cache.append(0, d[:, 3:5], d[:, 5:7], _ids(1, 0), _ids(*starts))
        torch.cuda.synchronize()
        assert int(cache.status.item()) & 4
        cache.status.zero_()
    cache.append(0, d[:1, 3:5], d[:1, 5:7], _ids(5))
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()
    for a, b in zip(before[:1], (cache.k,)):
        assert a.shape == b.shape


# ----------------------------------------------------------------- attention
def _check(cache, model, rng, rows, counts, heads, layer=0, starts=True, size=1.0, **kw):
    total = sum(counts)
    q = _bf16(rng, total, heads, cache.head_dim, size=size)
    at = [0] + [int(x) for x in np.cumsum(counts)]
    args = (layer, q.cuda(), _ids(*rows), _ids(*at) if starts else None)
    more = dict(max_new=max(counts)) if starts else {}
    got, lse = cache.attend(*args, lse=True, **more, **kw)
    got2, lse2 = cache.attend(*args, lse=True, **more, **kw)
    kw.pop("max_len", None)
    out, ref, slack, spread = model.attend(layer, _f64(q), rows, at, **kw)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    assert torch.equal(got, got2) and torch.equal(lse, lse2)
    g, l = _f64(got), _f64(lse)
    empty = np.isneginf(ref)
    assert np.array_equal(empty, np.isneginf(l)) and np.all(g[empty] == 0)
    assert np.all(np.abs(g - out) <= S.attend_bound(out, slack, spread)), float(np.abs(g - out).max())
    assert np.all(np.abs(l - ref)[~empty] <= slack[~empty] + 2.0 ** -20 * (1 + np.abs(ref[~empty])))
    return got


SHAPES = [  # head_dim, page, kv_heads, heads, rows' lengths
    (64, 16, 1, 1, [1]),
    (64, 64, 2, 4, [1, 15, 16, 17, 63, 64, 65]),
    (128, 32, 2, 10, [200, 1, 511]),
    (256, 16, 1, 2, [777, 128]),
    (80, 64, 2, 32, [100, 33]),
    (192, 128, 1, 3, [129, 300]),
    (1, 16, 1, 5, [70]),
    (96, 256, 1, 24, [255, 257, 3]),
    (33, 16, 3, 3, [90]),
]


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page,kv_heads,heads,lens", SHAPES, ids=[f"d{s[0]}_p{s[1]}_h{s[3]}of{s[2]}" for s in SHAPES])
def test_attention_of_single_tokens(dtype, dim, page, kv_heads, heads, lens):
    print("attend", dtype, dim, page, kv_heads, heads, lens, flush=True)
    rng = np.random.default_rng(dim + page + heads)
    n = len(lens)
    cache, model = _pair(layers=2, kv_heads=kv_heads, head_dim=dim, n_pages=sum(-(-x // page) for x in lens) + 3, max_seqs=n + 1,
                         max_pages=max(-(-x // page) for x in lens) + 1, page_tokens=page, dtype=dtype)
    _fill(cache, model, rng, list(range(n)), lens, (1.0, 3.0))
    for layer in (0, 1):
        for kw in ({}, dict(window=5), dict(window=64, sinks=3), dict(softcap=20.0), dict(scale=-0.3),
                   dict(window=1, sinks=200, softcap=50.0), dict(max_len=max(lens))):
            _check(cache, model, rng, list(range(n))[::-1], [1] * n, heads, layer, starts=False, **kw)


CHUNKS = [  # head_dim, page, kv_heads, heads, lengths, new tokens
    (64, 16, 1, 1, [5], [5]),
    (128, 64, 2, 4, [70, 300], [70, 33]),
    (128, 32, 1, 5, [400, 7, 64], [130, 1, 64]),
    (256, 16, 2, 4, [200, 90], [17, 90]),
    (64, 64, 1, 2, [260], [260]),
    (80, 16, 1, 40, [50], [19]),
    (192, 64, 2, 2, [150], [129]),
]


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page,kv_heads,heads,lens,new", CHUNKS, ids=[f"d{s[0]}_p{s[1]}_h{s[3]}of{s[2]}_n{max(s[5])}" for s in CHUNKS])
def test_attention_of_chunks(dtype, dim, page, kv_heads, heads, lens, new):
    print("attend chunk", dtype, dim, page, kv_heads, heads, lens, new, flush=True)
    rng = np.random.default_rng(dim + page + heads + max(new))
    n = len(lens)
    cache, model = _pair(layers=1, kv_heads=kv_heads, head_dim=dim, n_pages=sum(-(-x // page) for x in lens) + 3, max_seqs=n,
                         max_pages=max(-(-x // page) for x in lens) + 1, page_tokens=page, dtype=dtype)
    _fill(cache, model, rng, list(range(n)), lens)
    for kw in ({}, dict(window=30), dict(window=70, sinks=5, softcap=15.0), dict(window=3, sinks=1)):
        _check(cache, model, rng, list(range(n)), new, heads, **kw)


def test_rows_that_see_nothing():
    """An empty row, and more queries than the row has tokens: zeros and -infinity."""
    rng = np.random.default_rng(12)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=4, max_seqs=3, max_pages=4, page_tokens=16, dtype="e4m3")
    _fill(cache, model, rng, [1], [3])
    _check(cache, model, rng, [0, 1, 2], [2, 7, 1], 2)
    _check(cache, model, rng, [0, 1, 2], [1, 1, 1], 2, starts=False, window=2)
    out = cache.attend(0, torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"), _ids(0, 1), _ids(0, 0, 0))
    assert out.shape == (0, 2, 64)


def test_large_logits_and_far_apart_scales():
    """Logits of hundreds (one token takes all), pages whose scales differ by 2^20."""
    rng = np.random.default_rng(13)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=128, n_pages=20, max_seqs=1, max_pages=16, page_tokens=16, dtype="int8")
    for size in (1.0, 30.0, 1e-4, 1000.0, 0.0, 1.0):
        _fill(cache, model, rng, [0], [33], (size,))
    _check(cache, model, rng, [0], [1], 4, starts=False)
    _check(cache, model, rng, [0], [40], 4, softcap=30.0)
    _check(cache, model, rng, [0], [9], 4, scale=0.01)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_long_rows_are_split(dtype):
    """Rows long enough to be split over workgroups, ragged, with and without
    the workspace, windows that leave few of the tiles."""
    rng = np.random.default_rng(14)
    lens = [9000, 70, 3001]
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=200, max_seqs=3, max_pages=160, page_tokens=64, dtype=dtype)
    _fill(cache, model, rng, [0, 1, 2], lens)
    for kw in ({}, dict(window=1000, sinks=4), dict(softcap=10.0), dict(max_len=9000)):
        _check(cache, model, rng, [0, 1, 2], [1, 1, 1], 8, starts=False, **kw)
        _check(cache, model, rng, [2, 0], [3, 2], 8, **kw)


@pytest.mark.parametrize("heads,new", [(4, 1), (16, 40)])
def test_without_a_workspace(heads, new):
    """The C call with no workspace: rows are not split, the results hold the same bound."""
    import ctypes as C
    from lossless_entropy_coding_amd import _lib as L
    rng = np.random.default_rng(heads)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=128, n_pages=60, max_seqs=2, max_pages=40, page_tokens=64, dtype="e4m3")
    _fill(cache, model, rng, [0, 1], [2300, 700])
    q = _bf16(rng, 2 * new, heads, 128)
    qd, out, starts, rows = q.cuda(), torch.zeros(2 * new, heads, 128, dtype=torch.bfloat16, device="cuda"), _ids(0, new, 2 * new), _ids(0, 1)
    a = L.KvAttendArgs(0, 2, heads, 2 * new, new, 0, rows.data_ptr(), starts.data_ptr(), qd.data_ptr(), out.data_ptr(), None,
                       heads * 128, heads * 128, 0.0, 0.0, 0, 0)
    assert L.lib().bs_kv_attend_work_bytes(C.byref(cache.c), C.byref(a)) > 0
    assert L.lib().bs_kv_attend_async(C.byref(cache.c), C.byref(a), None, 0, None) == L.BS_OK
    torch.cuda.synchronize()
    want, _, slack, spread = model.attend(0, _f64(q), [0, 1], [0, new, 2 * new])
    assert np.all(np.abs(_f64(out) - want) <= S.attend_bound(want, slack, spread))


def test_many_rows_of_many_lengths():
    """Blocks of rows that two, three and more workgroups share, whole ones
    between them, rows that see nothing, bad table entries elsewhere."""
    rng = np.random.default_rng(21)
    lens, new = [3000, 1, 900, 64, 2100, 0], [90, 70, 200, 1, 33, 3]
    cache, model = _pair(layers=1, kv_heads=2, head_dim=64, n_pages=120, max_seqs=6, max_pages=50, page_tokens=64, dtype="int8")
    _fill(cache, model, rng, [0, 1, 2, 3, 4], lens[:5])
    for kw in ({}, dict(window=500, sinks=70), dict(scale=-0.2), dict(softcap=9.0)):
        for _ in range(2):                          # the counters are back at zero
            _check(cache, model, rng, [0, 1, 2, 3, 4, 5], new, 6, **kw)
    cache.table[3, 0] = -7
    out = cache.attend(0, _bf16(rng, sum(new), 6, 64).cuda(), _ids(0, 1, 2, 3, 4, 5),
                       _ids(*([0] + [int(x) for x in np.cumsum(new)])), max_new=max(new))
    assert torch.isfinite(out.float()).all()
    with pytest.raises(RuntimeError, match="does not exist"):
        cache.check()


@pytest.mark.parametrize("new", [1, 30])
def test_rows_longer_than_said(new):
    rng = np.random.default_rng(31)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=150, max_seqs=2, max_pages=140, page_tokens=64, dtype="int8")
    _fill(cache, model, rng, [0, 1], [8500, 40])
    for max_len in (1, 300, 3000):
        for _ in range(2):
            _check(cache, model, rng, [0, 1], [new, new], 8, max_len=max_len)


def test_query_ranges_that_do_not_exist():
    rng = np.random.default_rng(32)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=10, max_seqs=2, max_pages=4, page_tokens=16, dtype="int8")
    _fill(cache, model, rng, [0, 1], [40, 20])
    for heads in (2, 64):                           # few and many rows
        q = _bf16(rng, 3, heads, 64).cuda()
        want = cache.attend(0, q, _ids(0, 1), _ids(0, 2, 3), max_new=3)
        for starts in ((0, 2, 4), (-1, 2, 3), (2, 0, 3), (0, 2, 1)):
            out = torch.zeros_like(q)
            cache.attend(0, q, _ids(0, 1), _ids(*starts), max_new=3, out=out)
            torch.cuda.synchronize()
            assert int(cache.status.item()) == 4
            cache.status.zero_()
            if starts[:2] == (0, 2):
                assert torch.equal(out[:2], want[:2])       # the other row is as it was


def test_children_share_and_diverge():
    """A forked row gives its parent's results, then both go their own ways; compaction moves neither."""
    rng = np.random.default_rng(15)
    cache, model = _pair(layers=2, kv_heads=2, head_dim=64, n_pages=30, max_seqs=5, max_pages=8, page_tokens=16, dtype="e4m3")
    _fill(cache, model, rng, [3, 0], [50, 16])
    cache.fork(_ids(3, 3, 0), _ids(1, 2, 4))
    model.fork([3, 3, 0], [1, 2, 4])
    _same(cache, model)
    got = _check(cache, model, rng, [3, 1, 2, 0, 4], [1] * 5, 4, layer=1, starts=False)
    assert got.shape[0] == 5
    _fill(cache, model, rng, [1, 2, 3, 4], [1, 20, 3, 1], (5.0,))
    _same(cache, model)
    cache.free(_ids(3))
    model.free([3])
    cache.compact()
    model.compact()
    _same(cache, model)
    _check(cache, model, rng, [1, 2, 0, 4], [1] * 4, 4, layer=1, starts=False)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes a side, used at its far end in its last layer."""
    rng = np.random.default_rng(16)
    cache = kv.KvCache(layers=3, kv_heads=8, head_dim=256, n_pages=12000, max_seqs=2, max_pages=8, page_tokens=64, dtype="int8")
    assert cache.k.numel() > 1 << 32
    model = S.Cache(layers=1, kv_heads=8, head_dim=256, n_pages=6, max_seqs=2, max_pages=8, page_tokens=64, dtype="int8")
    first = 11994
    cache.refs[:first] = 1
    cache.extend(_ids(0, 1), _ids(130, 65))
    model.extend([0, 1], [130, 65])
    assert torch.equal(cache.table[0, :3].cpu(), torch.from_numpy(model.table[0, :3]) + first)
    k, v = _bf16(rng, 195, 8, 256), _bf16(rng, 195, 8, 256)
    cache.append(2, k.cuda(), v.cuda(), _ids(0, 1), _ids(0, 130, 195))
    model.append(0, _f64(k), _f64(v), [0, 1], [0, 130, 195])
    for n in ("k", "v", "scale"):
        used = sorted(set(model.table[0, :3]) | set(model.table[1, :2]))
        a, b = getattr(cache, n)[2, first:].cpu().numpy()[used], getattr(model, n)[0][used]
        assert a.tobytes() == b.tobytes(), n
    q = _bf16(rng, 2, 16, 256)
    got, lse = cache.attend(2, q.cuda(), _ids(0, 1), lse=True)
    out, ref, slack, spread = model.attend(0, _f64(q), [0, 1])
    assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))
    cache.free(_ids(1))
    cache.fork(_ids(0), _ids(1))
    torch.cuda.synchronize()
    a, b = int(cache.table[0, 2]), int(cache.table[1, 2])
    assert a != b and all(torch.equal(getattr(cache, n)[:, a], getattr(cache, n)[:, b]) for n in ("k", "v", "scale"))
    cache.check()


def test_strided_queries_and_results():
    rng = np.random.default_rng(17)
    cache, model = _pair(layers=1, kv_heads=2, head_dim=72, n_pages=12, max_seqs=2, max_pages=8, page_tokens=16, dtype="e4m3")
    _fill(cache, model, rng, [0, 1], [100, 20])
    for off in (0, 1):
        buf = torch.zeros(off + 5 * 9 * 72, dtype=torch.bfloat16, device="cuda")[off:].view(5, 9, 72)
        q = _bf16(rng, 5, 4, 72)
        buf[:, 2:6] = q.cuda()
        res = torch.full((5, 6, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        got = cache.attend(0, buf[:, 2:6], _ids(0, 1), _ids(0, 3, 5), out=res[:, 1:5])
        out, ref, slack, spread = model.attend(0, _f64(q), [0, 1], [0, 3, 5])
        assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))
        assert bool((res[:, 0] == 7).all()) and bool((res[:, 5] == 7).all())


def test_graph_of_a_decode_step():
    """extend, append and attend captured once and replayed; each replay
    continues where the last ended and equals the eager step."""
    rng = np.random.default_rng(18)
    kw = dict(layers=2, kv_heads=2, head_dim=64, n_pages=80, max_seqs=4, max_pages=20, page_tokens=16, dtype="int8")
    cache, model = _pair(**kw)
    _fill(cache, model, rng, [0, 1, 2, 3], [31, 200, 1, 64])
    rows, ones = _ids(0, 1, 2, 3), _ids(1, 1, 1, 1)
    k, v = (torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, out = (torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(c):
        c.extend(rows, ones)
        for layer in range(2):
            c.append(layer, k[layer], v[layer], rows)
            c.attend(layer, q[layer], rows, out=out[layer])
    twin = kv.KvCache(**kw)
    for n in ("k", "v", "scale", "refs", "table", "lens"):
        getattr(twin, n).copy_(getattr(cache, n))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step(twin)                                   # workspaces are made before the capture
    torch.cuda.synchronize()
    for n in ("k", "v", "scale", "refs", "table", "lens"):
        getattr(twin, n).copy_(getattr(cache, n))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(twin)
    for n in range(5):
        for t in (k, v, q):
            t.copy_(_bf16(rng, *t.shape))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(cache)
        torch.cuda.synchronize()
        assert torch.equal(got, out), n
        for name in ("k", "v", "scale", "refs", "table", "lens"):
            assert getattr(twin, name).cpu().numpy().tobytes() == getattr(cache, name).cpu().numpy().tobytes(), (n, name)
    twin.check(), cache.check()


def test_work_on_another_stream():
    rng = np.random.default_rng(19)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=60, max_seqs=2, max_pages=50, page_tokens=64, dtype="e4m3")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        _fill(cache, model, rng, [0, 1], [2000, 5])
        q = _bf16(rng, 2, 4, 64)
        got = cache.attend(0, q.cuda(), _ids(0, 1))
    s.synchronize()
    out, ref, slack, spread = model.attend(0, _f64(q), [0, 1])
    assert np.all(np.abs(_f64(got) - out) <= S.attend_bound(out, slack, spread))
    _same(cache, model)


def test_a_call_on_another_stream_waits_for_nothing_on_this_one():
    rng = np.random.default_rng(33)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=130, max_seqs=2, max_pages=100, page_tokens=64, dtype="int8")
    _fill(cache, model, rng, [0, 1], [5000, 700])
    q, rows = _bf16(rng, 2, 4, 64).cuda(), _ids(0, 1)
    want = cache.attend(0, q, rows)
    fresh = kv.KvCache.over(cache.k, cache.v, cache.scale, cache.refs, cache.table, cache.lens, 64, "int8")
    full = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")
    a = torch.zeros(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    del full                                         # memory that is not zero, for whoever asks next
    for _ in range(20):
        a = a @ a                                    # keeps the current stream busy
    got = fresh.attend(0, q, rows, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()


def test_a_graph_outlives_a_larger_workspace():
    rng = np.random.default_rng(34)
    cache, model = _pair(layers=1, kv_heads=1, head_dim=64, n_pages=130, max_seqs=8, max_pages=100, page_tokens=64, dtype="e4m3")
    _fill(cache, model, rng, [0, 1], [3000, 2000])
    q, rows, out = _bf16(rng, 1, 4, 64).cuda(), _ids(0), torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        cache.attend(0, q, rows, out=out)
    torch.cuda.synchronize()
    small, want = cache._attend_work, out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.attend(0, q, rows, out=out)
    address = small.data_ptr()
    del small
    many = _ids(*([0, 1] * 40))
    cache.attend(0, _bf16(rng, 80, 32, 64).cuda(), many)
    assert cache._attend_work.data_ptr() != address
    others = [torch.full((1 << k,), 7, dtype=torch.uint8, device="cuda") for k in range(9, 22)]
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((t == 7).all()) for t in others)
