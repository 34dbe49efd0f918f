"""What the serving operators' Python calls hand to the library, on the CPU: a
stand-in takes the place of the library's launches, so no pointer is followed."""
import sys
import threading
import time

import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import _lib as L
from lossless_entropy_coding_amd import codec, kv, lora

LAUNCHES = ("bs_kv_extend_async", "bs_kv_fork_async", "bs_kv_compact_async", "bs_kv_append_async", "bs_kv_attend_async",
            "bs_kv_free_async", "bs_kv_copy_pages_async", "bs_lora_add_async", "bs_lora_batch_async",
            "bs_fixed_gemm_lora_async")


class Stub:
    """The library, except that its launches call `seen(name, args)`."""

    def __init__(self, seen):
        self._real, self._seen = L.lib(), seen

    def __getattr__(self, name):
        if name in LAUNCHES:
            return lambda *args: self._seen(name, args) or 0
        return getattr(self._real, name)


@pytest.fixture
def stub(monkeypatch):
    def start(seen):
        lib = Stub(seen)
        monkeypatch.setattr(L, "lib", lambda: lib)
        for m in (kv, lora, codec):
            monkeypatch.setattr(m, "_stream_of", lambda device, stream: 0)
    return start


def _run(*workers):
    """Each worker in a thread of its own, switched as often as they can be."""
    failed, old = [], sys.getswitchinterval()

    def guard(f):
        try:
            f()
        except BaseException as e:                   # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=guard, args=(w,)) for w in workers]
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    if failed:
        raise failed[0]


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_threads_that_attend_over_one_cache_send_their_own_arguments(stub):
    """The library reads its arguments after it has let other threads run."""
    sent = {}

    def seen(name, args):
        time.sleep(2e-5)
        a = args[1]._obj
        sent[threading.get_ident()].append((a.layer, a.total_q, a.d_seqs, a.d_q, a.d_out, a.d_lse, a.window, args[2], args[3]))
    stub(seen)
    cache = kv.KvCache(4, 1, 64, 16, 8, 400, device="cpu")

    def worker(i):
        def go():
            sent[threading.get_ident()] = mine = []
            q, rows, out, lse = _bf16(i + 1, 4, 64), torch.zeros(i + 1, dtype=torch.int32), _bf16(i + 1, 4, 64), torch.zeros(i + 1, 4)
            for _ in range(200):
                cache.attend(i, q, rows, window=i, out=out, lse=lse)
                got = mine.pop()
                assert got[:7] == (i, i + 1, rows.data_ptr(), q.data_ptr(), out.data_ptr(), lse.data_ptr(), i)
                assert got[7] is None or got[8] > 0
        return go
    _run(*[worker(i) for i in range(4)])


def test_calls_that_share_a_workspace_enqueue_their_launches_one_after_another(stub, monkeypatch):
    """A call of two launches must not have another's between them: both would
    use the one workspace."""
    inside = {}

    def seen(name, args):
        key = "page" if name in ("bs_kv_extend_async", "bs_kv_fork_async", "bs_kv_compact_async") else name
        assert not inside.get(key), name
        inside[key] = True
        time.sleep(2e-5)
        inside[key] = False
    stub(seen)
    monkeypatch.setattr(lora.LoraBatch, "update", lambda self, of, stream=None: None)
    cache = kv.KvCache(1, 1, 64, 16, 8, 4, device="cpu")
    ads = [(_bf16(4, 2048), _bf16(32, 4), 1.0)]
    pack = lora.LoraPack(ads, device="cpu")
    plan = codec.FixedPlan(codec.fixed_encode(np.full(32 * 2048, 0x3F80, np.uint16)), device="cpu")
    ids = torch.zeros(2, dtype=torch.int32)

    def pages():
        for _ in range(100):
            cache.extend(ids, ids), cache.fork(ids, ids), cache.compact(), cache.attend(0, _bf16(2, 1, 64), ids)

    def products():
        for n in range(1, 51):
            batch = lora.LoraBatch(torch.zeros(n, dtype=torch.int32), 1)
            pack.add(torch.zeros(n, 32), _bf16(n, 2048), batch)
            plan.gemm_lora(_bf16(n, 2048), 32, 2048, pack, batch)

    _run(pages, pages, products, products)


def test_counters_zeroed_in_a_capture_serve_no_other_call(stub, monkeypatch):
    """A recorded fill has not run when the next call is made."""
    given = []
    stub(lambda name, args: given.append((args[2], args[3])))
    cache = kv.KvCache(1, 1, 64, 16, 8, 400, device="cpu")
    q, ids = _bf16(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    recording = [True]
    monkeypatch.setattr(kv, "_capturing", lambda device: recording[0], raising=False)
    made, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    cache.attend(0, q, ids)
    cache.attend(0, q, ids)
    assert cache._attend_work is None and given[0][1] > 4096
    of = {t.data_ptr(): t for t in made}
    assert given[0][0] != given[1][0]
    for at, size in given:
        assert of[at].numel() == size and not of[at][:4096].any()
    recording[0] = False
    cache.attend(0, q, ids)
    w = cache._attend_work
    assert given[2][0] == w.data_ptr() and not w[:4096].any()
    recording[0] = True                              # large enough and zeroed before: captured calls take it, too
    cache.attend(0, q, ids)
    assert given[3][0] == w.data_ptr()
    q, ids = _bf16(8, 64, 64), torch.zeros(8, dtype=torch.int32)
    cache.attend(0, q, ids)
    assert given[4][1] > w.numel() and given[4][0] != w.data_ptr() and cache._attend_work is w


def _away(t):
    return t.to("meta")


def test_tensors_on_another_device_are_refused(stub):
    """Every argument in turn on a device that is not the cache's, the pack's
    or the plan's: nothing reaches the library."""
    launched = []
    stub(lambda name, args: launched.append(name))
    cache = kv.KvCache(1, 2, 64, 16, 8, 4, device="cpu")
    ids, starts = torch.zeros(2, dtype=torch.int32), torch.tensor([0, 1, 2], dtype=torch.int32)
    k, q, lse = _bf16(2, 2, 64), _bf16(2, 4, 64), torch.zeros(2, 4)
    pack = lora.LoraPack([(_bf16(4, 2048), _bf16(32, 4), 1.0)], device="cpu")
    plan = codec.FixedPlan(codec.fixed_encode(np.full(32 * 2048, 0x3F80, np.uint16)), device="cpu")
    batch = lora.LoraBatch(ids, 1)
    x, y = _bf16(2, 2048), torch.zeros(2, 32)
    calls = [
        (cache.extend, dict(rows=ids, counts=ids)), (cache.fork, dict(parents=ids, children=ids)), (cache.free, dict(rows=ids)),
        (cache.copy_pages, dict(source=ids, target=ids)),
        (cache.compact, dict(table_out=cache.table.clone(), refs_out=cache.refs.clone())),
        (cache.append, dict(layer=0, k=k, v=k, rows=ids, starts=starts)),
        (cache.attend, dict(layer=0, q=q, rows=ids, starts=starts, out=q.clone(), lse=lse)),
        (pack.add, dict(y=y, x=x, batch=batch, out=y.clone())), (batch.update, dict(adapter_of=ids)),
        (plan.gemm_lora, dict(x=x, rows=32, cols=2048, pack=pack, batch=batch, out=y)),
    ]
    for call, args in calls:
        del launched[:]
        call(**args, stream=None)
        assert len(launched) == 1, call
        for name in [n for n, v in args.items() if isinstance(v, torch.Tensor)]:
            with pytest.raises(ValueError, match="meta|on cpu"):
                call(**{**args, name: _away(args[name])})
            assert len(launched) == 1, (call, name)
    far = lora.LoraPack([(_bf16(4, 2048), _bf16(32, 4), 1.0)], device="cpu")
    far.a, far.device = _away(far.a), torch.device("meta")
    other = lora.LoraBatch(ids, 1)
    other.dev = _away(other.dev)
    del launched[:]
    for args in (dict(pack=far, batch=batch), dict(pack=pack, batch=other)):
        with pytest.raises(ValueError, match="meta"):
            plan.gemm_lora(x, 32, 2048, **args)
    with pytest.raises(ValueError, match="meta"):
        pack.add(y, x, other)
    parts = dict(k=cache.k, v=cache.v, scale=cache.scale, refs=cache.refs, table=cache.table, lens=cache.lens)
    kv.KvCache.over(**parts, head_dim=64)
    for name in parts:
        with pytest.raises(ValueError, match="meta|on cpu"):
            kv.KvCache.over(**{**parts, name: _away(parts[name])}, head_dim=64)
    assert not launched


def test_a_refused_attention_leaves_later_ones_their_workspace(stub):
    """The library's own checks, with nothing launched where they pass."""
    given = []
    real = L.lib()

    def seen(name, args):
        a = args[1]._obj
        if a.layer >= 2 or a.softcap < 0 or a.out_stride < 256:
            return real.bs_kv_attend_async(*args)
        given.append(args[3])
        return 0
    stub(seen)
    cache = kv.KvCache(2, 1, 64, 16, 8, 400, device="cpu")
    q, ids = _bf16(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(layer=9), dict(layer=0, softcap=-1.0), dict(layer=0, out=_bf16(4, 64).expand(2, 4, 64))):
        with pytest.raises(L.BSError):
            cache.attend(q=q, rows=ids, **bad)
    cache.attend(1, q, ids)
    cache.attend(0, q, ids)
    assert len(given) == 2 and given[0] == given[1] > 4096


def test_numbers_past_32_bits_keep_their_meaning(stub):
    """A window of 2^32 tokens is all of them, not none of its high bits; a layer of 2^32 is no layer."""
    given, real = [], L.lib()

    def seen(name, args):
        if (args[1] if name == "bs_kv_append_async" else args[1]._obj.layer) >= 2:
            return getattr(real, name)(*args)            # refused
        given.append(args)
    stub(seen)
    cache = kv.KvCache(2, 1, 64, 16, 8, 4, device="cpu")
    q, ids = _bf16(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    for big in (1 << 32, (1 << 32) + 5, 1 << 70):
        cache.attend(0, q, ids, window=big, sinks=big, max_len=big)
        a = given.pop()[1]._obj
        assert a.window == a.sinks == a.max_len == (1 << 32) - 1
        for layer in (big, -big, -1, 2):
            with pytest.raises(L.BSError, match="layer"):
                cache.attend(layer, q, ids)
            with pytest.raises(L.BSError, match="layer"):
                cache.append(layer, _bf16(2, 1, 64), _bf16(2, 1, 64), ids)
    assert not given
