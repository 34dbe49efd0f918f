"""Corners of the operators for several continuations that need no GPU: buffers
that lie over each other, workspaces, the references at the ends of a type."""
import ctypes as C
import math
import threading

import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import _lib as L
from lossless_entropy_coding_amd import kv
from oracle import serving as S
from test_branches_host import AT, PLAN, _attend, _cache, _plan


# --------------------------------------------------------------------- beams
@pytest.mark.parametrize("value", [-3.4e38, 3.4e38, 1e12, 0.0])
def test_the_reference_keeps_scores_beside_large_logits(value):
    """A row of one value is uniform over its tokens, whatever the value is."""
    x = np.full((2, 50), value)
    x[1] = np.linspace(-1, 1, 50)
    out, tok, par, _, _, _ = S.select(x, np.array([-5.0, -40.0]), 2, 3)
    np.testing.assert_allclose(out, [[-5.0 - math.log(50)] * 3], rtol=1e-12)
    assert tok.tolist() == [[0, 1, 2]] and par.tolist() == [[0, 0, 0]]


# --------------------------------------------------------------------- plans
BUFFERS = [n for n in PLAN if n.startswith("d_")]


@pytest.mark.parametrize("name", BUFFERS)
@pytest.mark.parametrize("which", ["rows", "counts", "groups"])
def test_inputs_that_are_the_plans_own_buffers(name, which):
    """From a buffer's first byte on; only the plan's own rows may be given as rows."""
    if (name, which) == ("d_rows", "rows"):
        return
    args = {"rows": AT, "counts": AT + 256, "groups": AT + 512, which: PLAN[name]}
    assert L.lib().bs_kv_batch_async(C.byref(_cache()), C.byref(_plan()), *args.values(), None) == L.BS_E_INVAL
    # nor do the rows make it right that another input is there, too
    if which != "rows":
        args["rows"] = PLAN["d_rows"]
        assert L.lib().bs_kv_batch_async(C.byref(_cache()), C.byref(_plan()), *args.values(), None) == L.BS_E_INVAL


@pytest.mark.parametrize("name", BUFFERS)
def test_plans_whose_buffers_lie_over_others(name):
    """Over each other, or over what the call reads of the cache."""
    f, cache = L.lib().bs_kv_batch_async, _cache(d_table=AT + 32768, d_lens=AT + 40960)
    sizes = {"d_rows": 12, "d_starts": 16, "d_places": 20, "d_slots": 40, "d_table": 48, "d_lead": 12, "d_shared": 12, "d_info": 176}
    for other in BUFFERS:
        if other != name:
            last = PLAN[other] + (sizes[other] - 1) // 16 * 16
            for at in (PLAN[other], last):
                assert f(C.byref(cache), C.byref(_plan(**{name: at})), AT, AT + 256, AT + 512, None) == L.BS_E_INVAL, (other, at)
    for at in (AT + 32768, AT + 32768 + 48, AT + 40960):         # 4 rows of 4 pages, 4 lengths
        assert f(C.byref(cache), C.byref(_plan(**{name: at})), AT, AT + 256, AT + 512, None) == L.BS_E_INVAL, at


# ------------------------------------------------------- attention of groups
@pytest.mark.parametrize("name", BUFFERS)
@pytest.mark.parametrize("many", [False, True])
def test_workspaces_that_lie_over_the_plan(name, many):
    lib, cache = L.lib(), _cache(max_pages=4096)
    at = dict(total=40, max_new=32) if many else {}
    plan = _plan(**at)
    need, work = int(lib.bs_kv_attend_shared_work_bytes(C.byref(cache), C.byref(_attend()), C.byref(plan))), 1 << 40
    assert need > 4096
    bad = _plan(**at, **{name: work + 4096})
    assert lib.bs_kv_attend_shared_async(C.byref(cache), C.byref(_attend()), C.byref(bad), work, need, None) == L.BS_E_INVAL


@pytest.mark.parametrize("rows", [1, 7, 512, 4096])
@pytest.mark.parametrize("pages", [1, 100, 8192])
def test_no_groups_need_no_more_workspace_than_one(rows, pages):
    lib, cache = L.lib(), _cache(kv_heads=8, head_dim=128, max_pages=pages)
    args = _attend(heads=40, q_stride=5120, out_stride=5120)
    need = [int(lib.bs_kv_attend_shared_work_bytes(C.byref(cache), C.byref(args), C.byref(_plan(n_seqs=rows, total=rows, max_new=1, n_groups=n))))
            for n in (0, 1)]
    assert 4096 < need[0] <= need[1]


# ------------------------------------------------------------------- threads
def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("name", ["bs_kv_batch_async", "bs_kv_append_async", "bs_kv_free_async", "bs_kv_copy_pages_async", "bs_kv_extend_async"])
def test_no_call_comes_between_a_compaction_and_its_table(name, monkeypatch):
    """Another thread's call is enqueued before the pages move, or after the cache has their new table."""
    real, seen, late = L.lib(), [], []

    class Stub:
        def __getattr__(self, f):
            if f == "bs_kv_compact_async":
                def compact(*args):
                    late.append(threading.Thread(target=calls[name]))
                    late[0].start()
                    late[0].join(0.2)
                    return 0
                return compact
            if f.startswith("bs_kv_") and f.endswith("_async"):
                return lambda cache, *args: seen.append((f, cache._obj.d_table)) or 0
            return getattr(real, f)
    monkeypatch.setattr(L, "lib", lambda: Stub())
    monkeypatch.setattr(kv, "_stream_of", lambda device, stream: 0)
    cache = kv.KvCache(1, 1, 64, 16, 4, 4, page_tokens=16, device="cpu")
    plan, x = kv.KvBatch(cache, _i(0, 1)), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    calls = {"bs_kv_batch_async": lambda: plan.update(_i(0, 1)), "bs_kv_append_async": lambda: cache.append(0, x, x, _i(0, 1)),
             "bs_kv_free_async": lambda: cache.free(_i(0)), "bs_kv_copy_pages_async": lambda: cache.copy_pages(_i(0), _i(1)),
             "bs_kv_extend_async": lambda: cache.extend(_i(0), _i(1))}
    old = cache.table.data_ptr()
    cache.compact()
    late[0].join(10)
    assert cache.table.data_ptr() != old and seen[-1] == (name, cache.table.data_ptr())
