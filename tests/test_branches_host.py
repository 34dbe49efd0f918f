"""Refusals of the operators for several continuations of a prompt (moved rows,
plans, attention of groups, the choice of beams): host checks that need no GPU;
what their Python calls check and hand to the library; the plain references
against independent facts."""
import ctypes as C
import itertools
import math

import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import _lib as L
from lossless_entropy_coding_amd import beam, codec, kv
from oracle import serving as S

BUF = (C.c_uint8 * (1 << 20))()
AT = (C.addressof(BUF) + 255) // 256 * 256           # an aligned address; nothing is launched on it


def _cache(**kw):
    d = dict(layers=2, n_pages=8, max_seqs=4, max_pages=4, kv_heads=2, head_dim=64, page_tokens=16, type=1, d_k=AT, d_v=AT,
             d_scale=AT, d_refs=AT, d_table=AT, d_lens=AT, d_status=None)
    d.update(kw)
    return L.KvCache(*[d[n] for n, _ in L.KvCache._fields_])


# ------------------------------------------------------------------- reorder
def test_moves_that_are_refused():
    lib, c = L.lib(), _cache()
    need = int(lib.bs_kv_reorder_work_bytes(C.byref(c), 3))
    assert need >= 4 * (2 + 18 + 4) and lib.bs_kv_reorder_work_bytes(C.byref(c), 4097) == 0
    assert lib.bs_kv_reorder_work_bytes(C.byref(_cache(page_tokens=8)), 3) == 0
    f, w = lib.bs_kv_reorder_async, AT + 4096
    for args in ((3, None, AT, w, need), (3, AT, None, w, need), (3, AT + 2, AT, w, need), (3, AT, AT + 1, w, need), (3, AT, AT, None, need),
                 (3, AT, AT, w + 4, need), (3, AT, AT, w, need - 1), (4097, AT, AT, w, 1 << 20), (3, w + 8, AT, w, need),
                 (3, AT, w + need - 4, w, need)):
        assert f(C.byref(c), *args, None) == L.BS_E_INVAL, args
    assert f(C.byref(_cache(layers=0)), 3, AT, AT, w, need, None) == L.BS_E_INVAL
    assert f(C.byref(c), 0, None, None, None, 0, None) == L.BS_OK


# --------------------------------------------------------------------- plans
PLAN = dict(n_seqs=3, n_groups=2, total=5, max_new=2, width=4, reserved=0, **{n: AT + 1024 * (i + 1) for i, n in enumerate(
    ("d_rows", "d_starts", "d_places", "d_slots", "d_table", "d_lead", "d_shared", "d_info"))})


def _plan(**kw):
    return L.KvBatch(*[{**PLAN, **kw}[n] for n, _ in L.KvBatch._fields_])


BAD_PLAN = [dict(n_seqs=16385), dict(n_groups=16385), dict(total=1 << 31), dict(max_new=0), dict(max_new=6), dict(n_seqs=0), dict(reserved=1)] + \
    [{n: None} for n in PLAN if n.startswith("d_")] + [{n: AT + 16386} for n in PLAN if n.startswith("d_")] + [dict(d_slots=AT + 16388), dict(d_info=AT + 16392)]


@pytest.mark.parametrize("kw", BAD_PLAN, ids=lambda kw: "-".join(kw))
def test_plans_that_are_refused(kw):
    c, lib = _cache(), L.lib()
    assert lib.bs_kv_batch_async(C.byref(c), C.byref(_plan(**kw)), AT, AT, AT, None) == L.BS_E_INVAL
    a = _attend()
    assert lib.bs_kv_attend_shared_async(C.byref(c), C.byref(a), C.byref(_plan(**kw)), AT, 1 << 19, None) == L.BS_E_INVAL
    assert lib.bs_kv_attend_shared_work_bytes(C.byref(c), C.byref(a), C.byref(_plan(**kw))) == 0


def test_plan_calls_that_are_refused():
    c, f = _cache(), L.lib().bs_kv_batch_async
    assert f(C.byref(c), None, AT, AT, AT, None) == L.BS_E_INVAL
    assert f(C.byref(_cache(type=0)), C.byref(_plan()), AT, AT, AT, None) == L.BS_E_INVAL
    for args in ((None, AT, AT), (AT + 2, AT, AT), (AT, AT + 1, AT), (AT, AT, AT + 2), (AT, None, AT), (AT, AT, None), (AT, AT, AT + 1020)):
        assert f(C.byref(c), C.byref(_plan()), *args, None) == L.BS_E_INVAL, args
    for name in PLAN:                                            # inputs in the plan's own buffers
        if name.startswith("d_"):
            for at in range(3):
                args = [AT, AT + 256, AT + 512]
                args[at] = PLAN[name] + 4
                assert f(C.byref(c), C.byref(_plan()), *args, None) == L.BS_E_INVAL, (name, at)
    none = _plan(n_seqs=0, total=0, d_rows=None, d_starts=None, d_info=None)
    assert f(C.byref(c), C.byref(none), None, None, None, None) == L.BS_OK


# ------------------------------------------------------- attention of groups
def _attend(**kw):
    d = dict(layer=0, n_seqs=0, heads=4, total_q=0, max_new=0, max_len=0, d_seqs=None, d_starts=None, d_q=AT + 8192, d_out=AT + 16384,
             d_lse=None, q_stride=256, out_stride=256, scale=0.0, softcap=0.0, window=0, sinks=0)
    d.update(kw)
    return L.KvAttendArgs(*[d[n] for n, _ in L.KvAttendArgs._fields_])


def test_attention_of_groups_that_is_refused():
    lib, c, p = L.lib(), _cache(), _plan()
    need, w = int(lib.bs_kv_attend_shared_work_bytes(C.byref(c), C.byref(_attend()), C.byref(p))), AT + 65536
    assert need >= 4096 + 4 * 5 * 4 * 2 * 68

    def call(work=w, size=need, **kw):
        return lib.bs_kv_attend_shared_async(C.byref(c), C.byref(_attend(**kw)), C.byref(p), work, size, None)
    for kw in (dict(layer=2), dict(heads=3), dict(heads=0), dict(d_q=None), dict(d_out=None), dict(d_q=AT + 8193), dict(d_out=AT + 1),
               dict(d_lse=AT + 2), dict(q_stride=255), dict(out_stride=255), dict(softcap=-1.0), dict(softcap=math.nan), dict(scale=math.nan),
               dict(work=None), dict(work=w + 8), dict(size=need - 1), dict(d_q=w + 64), dict(d_out=w + need - 2), dict(d_lse=w)):
        assert call(**kw) == L.BS_E_INVAL, kw
    for name in ("d_rows", "d_starts", "d_places", "d_info"):
        q = _plan(**{name: w + 16})
        assert lib.bs_kv_attend_shared_async(C.byref(c), C.byref(_attend()), C.byref(q), w, need, None) == L.BS_E_INVAL, name
    assert lib.bs_kv_attend_shared_async(C.byref(c), None, C.byref(p), w, need, None) == L.BS_E_INVAL
    empty = _plan(n_seqs=0, total=0)
    assert lib.bs_kv_attend_shared_async(C.byref(c), C.byref(_attend()), C.byref(empty), None, 0, None) == L.BS_OK
    # too many for a launch's threads
    big = _plan(n_seqs=16384, total=1 << 29, max_new=1 << 15)
    assert lib.bs_kv_attend_shared_work_bytes(C.byref(_cache(kv_heads=1024)), C.byref(_attend(heads=1024, q_stride=1 << 16, out_stride=1 << 16)),
                                              C.byref(big)) == 0


def test_many_rows_go_to_the_attention_of_rows():
    """From 64 rows of a key head on the workspace is that call's own."""
    lib, c = L.lib(), _cache(max_pages=4096, n_pages=8)
    p = _plan(total=40, max_new=32)
    a = _attend()
    b = _attend(n_seqs=3, total_q=40, max_new=32, d_seqs=AT, d_starts=AT)
    assert lib.bs_kv_attend_shared_work_bytes(C.byref(c), C.byref(a), C.byref(p)) == lib.bs_kv_attend_work_bytes(C.byref(c), C.byref(b)) > 0


# --------------------------------------------------------------------- beams
BEAM = dict(batch=2, beams=4, keep=5, vocab=300, type=L.T_BF16, eos=-1, softcap=0.0, reserved=0, row_stride=300, d_logits=AT, d_scores=AT + 8192,
            d_done=None, d_scores_out=AT + 9216, d_tokens=AT + 10240, d_parents=AT + 11264, d_done_out=AT + 12288)


def _beam(**kw):
    return L.BeamArgs(*[{**BEAM, **kw}[n] for n, _ in L.BeamArgs._fields_])


BAD_SHAPE = [dict(beams=0), dict(beams=65), dict(keep=0), dict(keep=129), dict(batch=20000), dict(vocab=0), dict(vocab=1000001), dict(type=0),
             dict(type=3), dict(row_stride=299), dict(softcap=-1.0), dict(softcap=math.nan), dict(reserved=1)]
BAD_CALL = [{n: None} for n in BEAM if n.startswith("d_") and n != "d_done"] + \
    [dict(d_logits=AT + 1), dict(type=L.T_FP32, d_logits=AT + 2), dict(d_scores=AT + 8194), dict(d_done=AT + 8193, eos=1), dict(d_done=AT + 13312),
     dict(d_tokens=AT + 10241), dict(d_scores_out=AT + 8192), dict(d_tokens=AT), dict(d_parents=AT + 10240), dict(d_done_out=AT + 13312, d_done=AT + 13312, eos=2)]


@pytest.mark.parametrize("kw", BAD_SHAPE + BAD_CALL, ids=lambda kw: "-".join(kw))
def test_choices_that_are_refused(kw):
    lib, w = L.lib(), AT + 65536
    need = int(lib.bs_beam_work_bytes(C.byref(_beam())))
    assert 4096 < need < 1 << 19
    assert (lib.bs_beam_work_bytes(C.byref(_beam(**kw))) == 0) == (kw in BAD_SHAPE)
    assert lib.bs_beam_select_async(C.byref(_beam(**kw)), w, 1 << 19, None) == L.BS_E_INVAL


def test_choices_without_a_workspace_are_refused():
    lib, w = L.lib(), AT + 65536
    need = int(lib.bs_beam_work_bytes(C.byref(_beam())))
    for work, size in ((None, need), (w + 8, need), (w, need - 1), (AT, need), (AT + 12288 - need + 4, need)):
        assert lib.bs_beam_select_async(C.byref(_beam()), work if work is None or work % 16 in (0, 8) else work // 16 * 16, size, None) == L.BS_E_INVAL
    assert lib.bs_beam_select_async(None, w, need, None) == L.BS_E_INVAL and lib.bs_beam_work_bytes(None) == 0
    assert lib.bs_beam_select_async(C.byref(_beam(batch=0)), None, 0, None) == L.BS_OK


@pytest.mark.parametrize("batch,beams,keep,vocab,kind", itertools.product((1, 64, 1000), (1, 64), (1, 128), (1, 1000, 1000000), (1, 2)))
def test_workspaces_hold_all_parts(batch, beams, keep, vocab, kind):
    """At most 64 parts of a row; each leaves 16 B and its best."""
    if batch * beams > 65535:
        return
    need = int(L.lib().bs_beam_work_bytes(C.byref(_beam(batch=batch, beams=beams, keep=keep, vocab=vocab, row_stride=vocab, type=kind))))
    best, per = min(keep, vocab), 512 * (8 if kind == L.T_BF16 else 4) * 8
    least = -(-vocab // per) * batch * beams * (16 + 8 * best)
    assert 4096 + least <= need <= 4096 + 64 * batch * beams * (16 + 8 * best) + 512


# ------------------------------------------------------------- Python's calls
LAUNCHES = ("bs_kv_reorder_async", "bs_kv_batch_async", "bs_kv_attend_shared_async", "bs_beam_select_async")


@pytest.fixture
def calls(monkeypatch):
    real, seen = L.lib(), []

    class Stub:
        def __getattr__(self, name):
            if name in LAUNCHES:
                return lambda *args: seen.append((name, args)) or 0
            return getattr(real, name)
    monkeypatch.setattr(L, "lib", lambda: Stub())
    for m in (kv, beam, codec):
        monkeypatch.setattr(m, "_stream_of", lambda device, stream: 0)
    return seen


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_what_the_plan_checks_and_sends(calls):
    cache = kv.KvCache(1, 2, 64, 16, 8, 8, page_tokens=16, device="cpu")
    b = kv.KvBatch(cache, _i(0, 1, 2), _i(1, 2, 3), groups=_i(0, 2, 3), total=6, max_new=3, max_len=50)
    assert b.starts.numel() == 4 and b.places.numel() == b.slots.numel() == 6 and b.slots.dtype == torch.int64 and b.table.shape == (3, 4)
    assert b.slots.data_ptr() % 8 == 0 and b._info.data_ptr() % 16 == 0 and b.n_groups == 2
    c = calls[-1][1][1]._obj
    assert (c.n_seqs, c.n_groups, c.total, c.max_new, c.width) == (3, 2, 6, 3, 4)
    one = kv.KvBatch(cache, _i(0, 1))
    assert (one.total, one.max_new, one.n_groups, one.table.shape) == (2, 1, 1, (2, 8)) and calls[-1][1][3:5] == (None, None)
    n = len(calls)
    with pytest.raises(ValueError, match="total"):
        kv.KvBatch(cache, _i(0, 1), _i(1, 1))
    for args, kw in (((_i(0, 1), _i(1, 2, 3)), dict(groups=_i(0, 2, 3))), ((_i(0, 1, 2), None), dict(groups=_i(0, 2, 3))),
                     ((_i(0, 1, 2), _i(1, 2)), dict(groups=_i(0, 2, 3))), ((_i(0, 1, 2), _i(1, 2, 3)), dict(groups=_i(0, 3))),
                     ((_i(0, 1, 2).long(), _i(1, 2, 3)), dict(groups=_i(0, 2, 3)))):
        with pytest.raises(ValueError):
            b.update(*args, **kw)
    with pytest.raises(ValueError):
        one.update(_i(0, 1), _i(1, 1))
    assert len(calls) == n
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    out, lse = cache.attend_shared(0, q, b, lse=True, window=7)
    name, args = calls[-1]
    assert name == "bs_kv_attend_shared_async" and out.shape == q.shape and lse.shape == (6, 4)
    assert args[1]._obj.d_q == q.data_ptr() and args[1]._obj.window == 7 and args[1]._obj.max_len == 50 and args[2]._obj.total == 6
    assert args[3] == cache._attend_work.data_ptr() and args[4] > 4096
    for bad in (q[:5], q.float(), torch.zeros(6, 4, 32, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            cache.attend_shared(0, bad, b)
    other = kv.KvCache(1, 2, 64, 16, 8, 8, page_tokens=16, device="cpu")
    with pytest.raises(ValueError, match="another"):
        other.attend_shared(0, q, b)
    for kw in (dict(window=-1), dict(sinks=-1), dict(out=q[:5]), dict(lse=torch.zeros(5, 4))):
        with pytest.raises(ValueError):
            cache.attend_shared(0, q, b, **kw)


def test_what_moves_check_and_send(calls):
    cache = kv.KvCache(1, 2, 64, 16, 8, 8, page_tokens=16, device="cpu")
    rows, parents = _i(3, 1), _i(1, 1)
    cache.reorder(rows, parents)
    assert calls[-1][0] == "bs_kv_reorder_async" and calls[-1][1][1:4] == (2, rows.data_ptr(), parents.data_ptr())
    assert calls[-1][1][5] >= L.lib().bs_kv_reorder_work_bytes(cache._ref, 2)
    for r, p in ((rows, _i(1)), (rows.long(), parents), (rows, parents.view(1, 2)), (rows, _i(1, 5, 1, 5)[::2])):
        with pytest.raises(ValueError):
            cache.reorder(r, p)


def test_what_the_choice_checks_and_sends(calls):
    b = beam.Beams(2, 3, keep=4, eos=7, device="cpu")
    x, s, d = torch.zeros(6, 50, dtype=torch.bfloat16), torch.zeros(2, 3), torch.zeros(6, dtype=torch.int32)
    got = b.select(x, s, done=d, softcap=30.0)
    a = calls[-1][1][0]._obj
    assert (a.batch, a.beams, a.keep, a.vocab, a.type, a.eos, a.softcap, a.row_stride) == (2, 3, 4, 50, L.T_BF16, 7, 30.0, 50)
    assert (a.d_logits, a.d_scores, a.d_done) == (x.data_ptr(), s.data_ptr(), d.data_ptr())
    assert (a.d_scores_out, a.d_tokens, a.d_parents, a.d_done_out) == tuple(t.data_ptr() for t in got)
    assert got.scores.dtype == torch.float32 and all(t.shape == (2, 4) for t in got)
    wide = torch.zeros(6, 64)[:, 3:53]
    b.select(wide, s)
    a = calls[-1][1][0]._obj
    assert (a.type, a.row_stride, a.d_done) == (L.T_FP32, 64, None)
    n = len(calls)
    for args, kw in (((x[:5], s), {}), ((x.half(), s), {}), ((x.T.contiguous().T, s), {}), ((x, s[:1]), {}), ((x, s.double()), {}),
                     ((x, s), dict(done=d.bool())), ((x, s), dict(done=d[:5])), ((x.view(2, 3, 50), s), {})):
        with pytest.raises(ValueError):
            b.select(*args, **kw)
    assert len(calls) == n
    for kw in (dict(beams=0), dict(beams=65), dict(keep=0), dict(keep=129), dict(batch=30000), dict(eos=1 << 31)):
        with pytest.raises(ValueError):
            beam.Beams(**{**dict(batch=2, beams=3, device="cpu"), **kw})


def test_vocabularies_past_32_bits_are_refused(calls):
    b = beam.Beams(1, 1, device="cpu")
    b.select(torch.empty(1, (1 << 32) + 5, dtype=torch.bfloat16), torch.zeros(1))        # memory that nothing touches
    assert calls[-1][1][0]._obj.vocab == (1 << 32) - 1 and L.lib().bs_beam_work_bytes(b._ref) == 0


# ---------------------------------------------------------------- references
def test_the_reference_of_the_choice_is_the_definition():
    """Against a full sort of all continuations of a small case, and known answers."""
    rng = np.random.default_rng(0)
    x, s = rng.standard_normal((6, 9)), rng.standard_normal(6)
    out, tok, par, done, gaps, _ = S.select(x, s, 3, 5)
    for b in range(2):
        every = []
        for w in range(3 * b, 3 * b + 3):
            p = np.exp(x[w]) / np.exp(x[w]).sum()
            every += [(-(s[w] + math.log(p[v])), w, v) for v in range(9)]
        every.sort()
        assert [(w, v) for _, w, v in every[:5]] == list(zip(par[b], tok[b]))
        np.testing.assert_allclose(out[b], [-e for e, _, _ in every[:5]], rtol=1e-12)
        np.testing.assert_allclose(gaps[b], [every[i + 1][0] - every[i][0] for i in range(5)], atol=1e-12)
    out, tok, par, done, _, _ = S.select(np.zeros((2, 4)), np.array([0.0, -np.inf]), 2, 6)       # ties, a dead beam, too few
    assert tok.tolist() == [[0, 1, 2, 3, -1, -1]] and par.tolist() == [[0, 0, 0, 0, -1, -1]] and np.isneginf(out[0, 4:]).all()
    np.testing.assert_allclose(out[0, :4], -math.log(4))
    out, tok, par, done, _, _ = S.select(np.zeros((2, 4)), np.array([0.0, -1.0]), 2, 2, done=[0, 1], eos=3)
    assert tok.tolist() == [[3, 0]] and par.tolist() == [[1, 0]] and done.tolist() == [[1, 0]] and out[0, 0] == -1.0


def test_the_reference_of_moves_keeps_every_token():
    rng = np.random.default_rng(1)
    m = S.Cache(1, 1, 4, 40, 6, 6, page_tokens=16, dtype="int8")
    m.k[:] = rng.integers(0, 256, m.k.shape)
    m.extend([0, 1, 2, 3], [20, 32, 5, 50])
    m.scale[:] = 1
    rows, parents = [3, 0, 2, 1, 5], [0, 0, 3, 1, -1]
    want = [m.tokens(0, rows[q], 0, 0).copy() if q >= 0 else np.zeros((0, 4)) for q in parents]
    m.reorder(rows, parents)
    for r, w in zip(rows, want):
        np.testing.assert_array_equal(m.tokens(0, r, 0, 0), w)
    assert int(m.refs.sum()) == sum(m.pages(n) for n in m.lens) and m.refs.min() == 0
    starts, places, slots, table, lead, shared = m.batch([3, 0, 2], [2, 1, 0], [0, 2, 3], 3, 4)
    assert starts.tolist() == [0, 2, 3, 3] and places.tolist() == [48, 49, 49] and lead.tolist() == [0, 0, 2]
    assert shared[0] == shared[1] == 0 and shared[2] == 0                           # 48 tokens in common: less than 64
    assert slots[0] == m.table[3, 3] * 16
