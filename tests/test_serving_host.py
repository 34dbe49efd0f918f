"""Refusals of the serving operators (adapters, the key/value cache) and their
sizes: host checks that need no GPU, and the plain references against
independent facts."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import _lib as L
from oracle import serving as S

BUF = (C.c_uint8 * 8192)()
AT = (C.addressof(BUF) + 255) // 256 * 256           # an aligned address; nothing is launched on it


def _cache(**kw):
    d = dict(layers=2, n_pages=8, max_seqs=4, max_pages=4, kv_heads=2, head_dim=64, page_tokens=16, type=1, d_k=AT, d_v=AT,
             d_scale=AT, d_refs=AT, d_table=AT, d_lens=AT, d_status=None)
    d.update(kw)
    return L.KvCache(*[d[n] for n, _ in L.KvCache._fields_])


BAD_CACHE = [dict(layers=0), dict(n_pages=0), dict(max_seqs=0), dict(max_pages=0), dict(kv_heads=0), dict(head_dim=0),
             dict(head_dim=257), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=512), dict(type=0), dict(type=3),
             dict(d_k=None), dict(d_v=None), dict(d_scale=None), dict(d_refs=None), dict(d_table=None), dict(d_lens=None),
             dict(d_k=AT + 8), dict(d_v=AT + 4), dict(d_refs=AT + 4), dict(max_pages=1 << 30), dict(d_status=AT + 2)]


@pytest.mark.parametrize("kw", BAD_CACHE, ids=[str(k) for k in BAD_CACHE])
def test_caches_that_are_refused(kw):
    c, lib = _cache(**kw), L.lib()
    assert lib.bs_kv_free_async(C.byref(c), 1, AT, None) == L.BS_E_INVAL
    assert lib.bs_kv_pages_work_bytes(C.byref(c), 1) == 0


def test_cache_sizes():
    c, s = _cache(head_dim=80, d_k=None), L.KvSizes()
    assert L.lib().bs_kv_sizes_get(C.byref(c), C.byref(s)) == L.BS_OK
    assert (s.wide, s.side_bytes, s.scale_bytes, s.page_bytes) == (128, 2 * 8 * 2 * 16 * 128, 2 * 8 * 2 * 8, 2 * 2 * 16 * 128 + 16)
    assert L.lib().bs_kv_sizes_get(C.byref(c), None) == L.BS_E_INVAL


def test_page_calls_that_are_refused():
    lib, c = L.lib(), _cache()
    w = int(lib.bs_kv_pages_work_bytes(C.byref(c), 2))
    assert w >= 4 * (1 + 8 + 4)
    for f in (lib.bs_kv_extend_async, lib.bs_kv_fork_async):
        assert f(C.byref(c), 2, None, AT, AT, w, None) == L.BS_E_INVAL
        assert f(C.byref(c), 2, AT, None, AT, w, None) == L.BS_E_INVAL
        assert f(C.byref(c), 2, AT, AT, None, w, None) == L.BS_E_INVAL
        assert f(C.byref(c), 2, AT, AT, AT + 4, w, None) == L.BS_E_INVAL
        assert f(C.byref(c), 2, AT, AT, AT, w - 1, None) == L.BS_E_INVAL
        assert f(C.byref(c), 70000, AT, AT, AT, 1 << 30, None) == L.BS_E_INVAL
        assert f(C.byref(c), 0, None, None, AT, w, None) == L.BS_OK                   # nothing to do
    assert lib.bs_kv_free_async(C.byref(c), 1, None, None) == L.BS_E_INVAL
    assert lib.bs_kv_copy_pages_async(C.byref(c), 1, AT, None, None) == L.BS_E_INVAL
    assert lib.bs_kv_copy_pages_async(C.byref(c), 0, None, None, None) == L.BS_OK
    w0 = int(lib.bs_kv_pages_work_bytes(C.byref(c), 0))
    f = lib.bs_kv_compact_async
    assert f(C.byref(c), None, AT + 1024, AT, w0, None) == L.BS_E_INVAL
    assert f(C.byref(c), AT, AT + 1024, AT + 2048, w0, None) == L.BS_E_INVAL          # the cache's own table
    assert f(C.byref(c), AT + 1024, AT, AT + 2048, w0, None) == L.BS_E_INVAL          # its own counts
    assert f(C.byref(c), AT + 1024, AT + 1040, AT + 2048, w0, None) == L.BS_E_INVAL   # each other
    assert f(C.byref(c), AT + 1024, AT + 1536, AT + 2048, w0 - 1, None) == L.BS_E_INVAL


def test_appends_that_are_refused():
    lib, c = L.lib(), _cache()
    ok = dict(layer=0, n=2, seqs=AT, starts=None, total=2, most=1, k=AT, ks=128, v=AT, vs=128, t=1)

    def call(**kw):
        a = {**ok, **kw}
        return lib.bs_kv_append_async(C.byref(c), a["layer"], a["n"], a["seqs"], a["starts"], a["total"], a["most"], a["k"],
                                      a["ks"], a["v"], a["vs"], a["t"], None)
    for kw in (dict(layer=2), dict(seqs=None), dict(k=None), dict(v=None), dict(ks=127), dict(vs=64), dict(t=0), dict(t=3),
               dict(k=AT + 1), dict(t=2, v=AT + 2), dict(total=3), dict(most=2), dict(most=0, starts=AT),
               dict(most=3, starts=AT), dict(n=70000, total=70000)):
        assert call(**kw) == L.BS_E_INVAL, kw
    assert call(n=0, total=0) == L.BS_OK and call(total=0, starts=AT) == L.BS_OK


def test_attentions_that_are_refused():
    lib, c = L.lib(), _cache()
    ok = dict(layer=0, n_seqs=2, heads=4, total_q=2, max_new=1, max_len=0, d_seqs=AT, d_starts=None, d_q=AT, d_out=AT,
              d_lse=None, q_stride=256, out_stride=256, scale=0.0, softcap=0.0, window=0, sinks=0)

    def args(**kw):
        a = {**ok, **kw}
        return L.KvAttendArgs(*[a[n] for n, _ in L.KvAttendArgs._fields_])
    for kw in (dict(layer=2), dict(heads=0), dict(heads=3), dict(total_q=3), dict(max_new=2), dict(d_seqs=None),
               dict(d_q=None), dict(d_out=None), dict(q_stride=255), dict(out_stride=128), dict(softcap=-1.0),
               dict(softcap=math.nan), dict(scale=math.nan), dict(d_q=AT + 1), dict(d_lse=AT + 2), dict(max_new=0),
               dict(d_starts=AT, max_new=3)):
        assert lib.bs_kv_attend_async(C.byref(c), C.byref(args(**kw)), None, 0, None) == L.BS_E_INVAL, kw
    assert lib.bs_kv_attend_async(C.byref(c), None, None, 0, None) == L.BS_E_INVAL
    assert lib.bs_kv_attend_async(None, C.byref(args()), None, 0, None) == L.BS_E_INVAL
    assert lib.bs_kv_attend_async(C.byref(c), C.byref(args(n_seqs=0, total_q=0)), None, 0, None) == L.BS_OK
    # a workspace that is given is checked
    big = _cache(max_pages=1 << 16, max_seqs=4)
    need = int(lib.bs_kv_attend_work_bytes(C.byref(big), C.byref(args())))
    assert need > 0
    assert lib.bs_kv_attend_async(C.byref(big), C.byref(args()), AT, need - 1, None) == L.BS_E_INVAL
    assert lib.bs_kv_attend_async(C.byref(big), C.byref(args()), AT + 4, need, None) == L.BS_E_INVAL


def _pack(**kw):
    d = dict(adapters=2, rank=16, rows=32, cols=64, d_a=AT, d_b=AT, d_ranks=AT, d_factor=AT)
    d.update(kw)
    return L.LoraPack(*[d[n] for n, _ in L.LoraPack._fields_])


def test_adapters_that_are_refused():
    lib = L.lib()
    bad = (dict(adapters=0), dict(adapters=4097), dict(rank=8), dict(rank=48), dict(rank=256), dict(rows=0), dict(cols=0),
           dict(rows=1 << 26), dict(d_a=None), dict(d_b=None), dict(d_ranks=None), dict(d_factor=None), dict(d_a=AT + 2),
           dict(d_b=AT + 8))
    for kw in bad:
        assert lib.bs_lora_work_bytes(C.byref(_pack(**kw)), 4) == 0, kw
        assert lib.bs_lora_add_async(C.byref(_pack(**kw)), AT, 4, AT, 64, AT, AT, 32, 2, AT, 1 << 20, None) == L.BS_E_INVAL, kw
    p = _pack()
    w = int(lib.bs_lora_work_bytes(C.byref(p), 4))
    ok = dict(batch=AT, t=4, x=AT, xs=64, yi=AT, yo=AT, ys=32, yt=2, w=AT, wb=w)

    def call(**kw):
        a = {**ok, **kw}
        return lib.bs_lora_add_async(C.byref(p), a["batch"], a["t"], a["x"], a["xs"], a["yi"], a["yo"], a["ys"], a["yt"],
                                     a["w"], a["wb"], None)
    for kw in (dict(batch=None), dict(x=None), dict(yi=None), dict(yo=None), dict(w=None), dict(xs=63), dict(ys=31),
               dict(yt=0), dict(yt=3), dict(wb=w - 1), dict(w=AT + 4), dict(yo=AT + 2), dict(t=(1 << 24) + 1)):
        assert call(**kw) == L.BS_E_INVAL, kw
    assert call(t=0) == L.BS_OK
    need = int(lib.bs_lora_batch_bytes(5, 2))
    assert need >= 4 * (4 + 4 * 3 + 5) and lib.bs_lora_batch_bytes(5, 0) == 0 and lib.bs_lora_batch_bytes(1 << 25, 1) == 0
    assert lib.bs_lora_batch_async(AT, 5, 2, AT, need - 1, None) == L.BS_E_INVAL
    assert lib.bs_lora_batch_async(None, 5, 2, AT, need, None) == L.BS_E_INVAL
    assert lib.bs_lora_batch_async(AT, 5, 2, None, need, None) == L.BS_E_INVAL
    assert lib.bs_lora_batch_async(AT, 5, 5000, AT, 1 << 20, None) == L.BS_E_INVAL


def test_products_with_adapters_that_are_refused():
    from lossless_entropy_coding_amd import codec
    lib = L.lib()
    blob = codec.fixed_encode(np.full(32 * 4096, 0x3F80, np.uint16))
    info, p = codec.fixed_info(blob), _pack(rows=32, cols=4096)
    f = lib.bs_fixed_gemm_lora_async
    w = int(lib.bs_fixed_gemm_lora_work_bytes(32, 4096, 4, C.byref(p)))
    assert w > 0 and lib.bs_fixed_gemm_lora_work_bytes(32, 4096, 65, C.byref(p)) == 0
    ok = dict(rows=32, cols=4096, n=4, x=AT, y=AT, pack=p, batch=AT, w=AT, wb=w)

    def call(**kw):
        a = {**ok, **kw}
        return f(C.byref(info), AT, a["rows"], a["cols"], a["n"], a["x"], a["y"], None, C.byref(a["pack"]), a["batch"],
                 a["w"], a["wb"], None)
    for kw in (dict(rows=64, cols=2048), dict(n=0), dict(n=65), dict(x=AT + 2), dict(x=None), dict(y=None), dict(batch=None),
               dict(w=None), dict(w=AT + 16), dict(wb=w - 1), dict(pack=_pack(rows=16, cols=4096)), dict(pack=_pack(rows=32))):
        assert call(**kw) == L.BS_E_INVAL, kw


def test_python_refusals():
    from lossless_entropy_coding_amd import kv, lora
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)   # noqa: E731
    for ads in ([], [(z(4, 8), z(6, 3), 1.0)], [(z(4, 8), z(6, 4), 1.0), (z(4, 9), z(6, 4), 1.0)], [(z(129, 8), z(6, 129), 1.0)],
                [(z(0, 8), z(6, 0), 1.0)]):
        with pytest.raises(ValueError):
            lora.LoraPack(ads, device="cpu")
    with pytest.raises(ValueError):
        kv.KvCache(1, 1, 300, 4, 1, 4, device="cpu")
    with pytest.raises(ValueError):
        kv.KvCache(1, 1, 64, 4, 1, 4, dtype="fp8", device="cpu")
    with pytest.raises(L.BSError):
        kv.KvCache(1, 1, 64, 4, 1, 4, page_tokens=24, device="cpu")
    c = kv.KvCache(1, 2, 64, 4, 2, 4, device="cpu")
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.extend(ids, ids[:1])
    with pytest.raises(ValueError):
        c.free(ids.long())
    with pytest.raises(ValueError):
        c.append(0, z(2, 2, 64), z(2, 2, 64, t=torch.bfloat16), ids)
    with pytest.raises(ValueError):
        c.append(0, z(2, 2, 32), z(2, 2, 32), ids)
    with pytest.raises(ValueError):
        c.append(0, z(3, 2, 64), z(3, 2, 64), ids)                            # three tokens for two rows, no starts
    with pytest.raises(ValueError):
        c.append(0, z(2, 64, 2).transpose(1, 2), z(2, 64, 2).transpose(1, 2), ids)
    with pytest.raises(ValueError):
        c.attend(0, z(2, 4, 64), ids)
    with pytest.raises(ValueError):
        c.attend(0, z(2, 4, 64, t=torch.bfloat16), ids, window=-1)
    with pytest.raises(ValueError):
        c.compact(table_out=c.table)


def test_reference_codes():
    v = S.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, t.astype(np.float64), equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 4001), np.random.default_rng(0).standard_normal(4000),
                        np.outer([1, -1], (v[:126] + v[1:127]) / 2).ravel()])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.round_to_code(x.astype(np.float32), "e4m3"), want)
    assert list(S.round_to_code(np.array([0.5, 1.5, -2.5, 126.5, 127]), "int8").view(np.int8)) == [0, 2, -2, 126, 127]
    for kind, q in S.LARGEST.items():
        assert S.scale_for(q, kind) == 1.0 and S.scale_for(np.nextafter(q, 999), kind) == 2.0 and S.scale_for(0.0, kind) == 2.0 ** -60


def test_workspace_sizes_of_refused_shapes_are_zero():
    lib, p = L.lib(), _pack(rows=32, cols=4096)
    size = lambda rows, cols, n=4, p=p: int(lib.bs_fixed_gemm_lora_work_bytes(rows, cols, n, C.byref(p)))   # noqa: E731
    assert size(32, 4096) > 0 and size(32, 4096, 64) > 0
    for shape in ((16, 4096), (32, 2048), (64, 2048), (1 << 60, 4096), (32, 1 << 60), (0, 4096), (32, 0), (32, 4096, 0)):
        assert size(*shape) == 0, shape
    for cols in (3584, 4095, 32, 2047):
        assert size(32, cols, 4, _pack(rows=32, cols=cols)) == 0, cols
    # 2^24 tokens of 2^26 - 1 rows: more workgroups than a launch takes
    assert lib.bs_lora_work_bytes(C.byref(_pack(rows=(1 << 26) - 1)), 1 << 24) == 0
    assert lib.bs_kv_pages_work_bytes(C.byref(_cache()), 65535) > 0 and lib.bs_kv_pages_work_bytes(C.byref(_cache()), 65536) == 0


def test_workspaces_over_inputs_or_results_are_refused():
    """Every part of a workspace, at its first and its last bytes.  Nothing is launched: the addresses are made up."""
    from lossless_entropy_coding_amd import codec
    lib, at, words = L.lib(), 1 << 30, 1 << 28           # buffers 256 MiB apart
    X, Y, W, O, B = at, at + words, at + 2 * words, at + 3 * words, at + 4 * words

    def refused(call, size, *others):
        for other, n in others:
            for w in (other, other + n // 256 * 256 - 256 if n >= 256 else other, (other - size) // 256 * 256 + 256):
                assert call(w) == L.BS_E_INVAL, (hex(w), hex(other), n, size)
    for rows, cols, n in ((32, 4096, 4), (32, 2048, 33), (64, 14336, 64), (4096, 2048, 1)):   # shares or none, X laid out or not
        blob = codec.fixed_encode(np.full(rows * cols, 0x3F80, np.uint16))
        info, p = codec.fixed_info(blob), _pack(rows=rows, cols=cols, d_a=B, d_b=B)
        size = int(lib.bs_fixed_gemm_lora_work_bytes(rows, cols, n, C.byref(p)))
        refused(lambda w: lib.bs_fixed_gemm_lora_async(C.byref(info), B, rows, cols, n, X, Y, None, C.byref(p), B, w, size, None),
                size, (X, 2 * n * cols), (Y, 4 * n * rows))
    p = _pack(rows=100, cols=200)
    size = int(lib.bs_lora_work_bytes(C.byref(p), 70))
    refused(lambda w: lib.bs_lora_add_async(C.byref(p), B, 70, X, 333, Y, O, 120, 1, w, size, None), size,
            (X, 2 * (69 * 333 + 200)), (Y, 2 * (69 * 120 + 100)), (O, 2 * (69 * 120 + 100)))
    c = _cache(max_pages=1 << 16, d_k=B, d_v=B)
    a = L.KvAttendArgs(*[dict(layer=0, n_seqs=2, heads=4, total_q=2, max_new=1, max_len=0, d_seqs=B, d_starts=None, d_q=X, d_out=Y,
                              d_lse=O, q_stride=300, out_stride=400, scale=0.0, softcap=0.0, window=0, sinks=0)[n]
                         for n, _ in L.KvAttendArgs._fields_])
    size = int(lib.bs_kv_attend_work_bytes(C.byref(c), C.byref(a)))
    refused(lambda w: lib.bs_kv_attend_async(C.byref(c), C.byref(a), w, size, None), size,
            (X, 2 * 556), (Y, 2 * 656), (O, 32))


def test_calls_of_more_threads_than_a_launch_takes_are_refused():
    """Up front and by name, not by the launch: a grid has less than 2^32 threads in x."""
    lib, big = L.lib(), _cache(kv_heads=8, max_pages=4096, max_seqs=4096, page_tokens=64)
    args = lambda **kw: L.KvAttendArgs(*[{**dict(layer=0, n_seqs=2048, heads=40, total_q=1 << 16, max_new=1 << 16, max_len=0, d_seqs=AT,   # noqa: E731
                                              d_starts=AT, d_q=AT, d_out=AT, d_lse=None, q_stride=40 * 64, out_stride=40 * 64, scale=0.0,
                                              softcap=0.0, window=0, sinks=0), **kw}[n] for n, _ in L.KvAttendArgs._fields_])
    for kw in (dict(), dict(n_seqs=1 << 23, total_q=1 << 23, max_new=16), dict(n_seqs=1 << 24, total_q=1 << 24, max_new=1, heads=40),
               dict(n_seqs=1 << 20, total_q=1 << 21, max_new=200, heads=8)):
        assert lib.bs_kv_attend_async(C.byref(big), C.byref(args(**kw)), None, 0, None) == L.BS_E_INVAL, kw
        assert b"too many" in lib.bs_last_error()
    assert lib.bs_kv_attend_work_bytes(C.byref(big), C.byref(args(n_seqs=4, total_q=256, max_new=64))) > 0
    wide = _cache(max_seqs=1 << 24, max_pages=1)
    w = int(lib.bs_kv_pages_work_bytes(C.byref(wide), 0))
    assert lib.bs_kv_compact_async(C.byref(wide), 1 << 40, 1 << 41, AT, w, None) == L.BS_E_INVAL
    # 2^24 tokens are 2^20 tiles and one begun for each adapter
    assert lib.bs_lora_work_bytes(C.byref(_pack(rows=15 * 1024)), 1 << 24) > 0
    assert lib.bs_lora_work_bytes(C.byref(_pack(rows=16 * 1024)), 1 << 24) == 0
