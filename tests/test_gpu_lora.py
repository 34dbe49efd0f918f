"""Low-rank adapters on the GPU against their definition in 64 bits.

The tolerance is the fp32 bound of oracle.serving.lora: every product of two
BF16 numbers is exact in fp32 and each addition rounds once; a result in BF16
is rounded once more (8 significant bits: by at most 2^-8 of it)."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import codec, lora
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _bf16(rng, *shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).bfloat16()


def _f64(t):
    return t.cpu().float().numpy().astype(np.float64)


def _adapters(rng, rows, cols, ranks):
    return [(_bf16(rng, r, cols, size=cols ** -0.5), _bf16(rng, rows, r, size=0.3), 0.25 + 0.5 * i)
            for i, r in enumerate(ranks)]


def _oracle(adapters):
    return [(_f64(a), _f64(b), s) for a, b, s in adapters]


CASES = [
    # rows, cols, ranks, the adapter of each token
    (1, 1, [1], [0]),
    (16, 32, [16], [0]),
    (33, 77, [3, 16, 1], [2, -1, 0, 0, 1]),
    (130, 65, [128, 5], [1] * 17 + [0] * 33 + [-1] * 3),
    (64, 4096, [33], [0] * 16),
    (257, 1000, [8, 64, 17, 40], [i % 5 - 1 for i in range(100)]),
    (96, 256, [16] * 40, list(range(40)) * 2),
    (48, 128, [4, 4], [-1] * 20),
    (4096, 512, [16], [0]),
    (500, 300, [20, 30], [0] * 700 + [1] * 321 + [-1] * 4),
]


@pytest.mark.parametrize("rows,cols,ranks,of", CASES, ids=[f"{c[0]}x{c[1]}_r{max(c[2])}_t{len(c[3])}" for c in CASES])
@pytest.mark.parametrize("y32", [True, False])
def test_add_matches_the_definition(rows, cols, ranks, of, y32):
    print("lora add", rows, cols, ranks, len(of), y32, flush=True)
    rng = np.random.default_rng(rows * 1000 + cols + len(of))
    ads = _adapters(rng, rows, cols, ranks)
    x, y = _bf16(rng, len(of), cols), torch.from_numpy(rng.standard_normal((len(of), rows)).astype(np.float32))
    y = y if y32 else y.bfloat16()
    ref, loose = S.lora(_f64(y), _f64(x), of, _oracle(ads))
    pack = lora.LoraPack(ads)
    batch = lora.LoraBatch(torch.tensor(of, dtype=torch.int32, device="cuda"), len(ads))
    yd = y.cuda()
    got = pack.add(yd, x.cuda(), batch, out=torch.full_like(yd, float("nan")))
    again = pack.add(yd, x.cuda(), batch, out=torch.full_like(yd, float("nan")))
    assert torch.equal(yd.cpu(), y) and torch.equal(got, again)
    tol = loose + (0 if y32 else 2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -8 * loose)
    assert np.all(np.abs(_f64(got) - ref) <= tol)
    assert pack.add(yd, x.cuda(), batch) is yd and torch.equal(yd, got)        # in place
    none = [t for t, a in enumerate(of) if a < 0]
    assert torch.equal(got.cpu()[none], y[none])
    assert batch.bad_indices() == 0


def test_strided_and_unaligned_rows():
    rng = np.random.default_rng(5)
    rows, cols, of = 70, 200, [0, 1, -1, 1, 0, 0, 1]
    ads = _adapters(rng, rows, cols, [9, 12])
    pack = lora.LoraPack(ads)
    batch = lora.LoraBatch(torch.tensor(of, dtype=torch.int32, device="cuda"), 2)
    for off, wide in ((0, 256), (1, 201), (3, 333), (8, 208)):
        xs = _bf16(rng, len(of), wide)[:, off if off + cols <= wide else 0:][:, :cols]
        ys = torch.from_numpy(rng.standard_normal((len(of), rows + 11)).astype(np.float32))
        xd, yd = xs.cuda(), ys.cuda()
        base = torch.zeros(len(of), wide, dtype=torch.bfloat16, device="cuda")
        o = off if off + cols <= wide else 0
        base[:, o:o + cols] = xd
        view, yv = base[:, o:o + cols], yd[:, 5:5 + rows]
        before = yd.clone()
        ref, loose = S.lora(_f64(yv), _f64(view), of, _oracle(ads))
        pack.add(yv, view, batch)
        assert np.all(np.abs(_f64(yv) - ref) <= loose)
        outside = torch.ones_like(yd, dtype=torch.bool)
        outside[:, 5:5 + rows] = False
        assert torch.equal(yd[outside], before[outside])


def test_bad_indices_count_as_none_and_no_tokens_do_nothing():
    rng = np.random.default_rng(6)
    ads = _adapters(rng, 20, 40, [4])
    pack = lora.LoraPack(ads)
    batch = lora.LoraBatch(torch.tensor([0, 1, -2, 1 << 30], dtype=torch.int32, device="cuda"), 1)
    x, y = _bf16(rng, 4, 40), torch.zeros(4, 20)
    got = pack.add(y.cuda(), x.cuda(), batch)
    assert batch.bad_indices() == 3
    assert float(got[1:].abs().max()) == 0 and float(got[0].abs().max()) > 0
    empty = lora.LoraBatch(torch.empty(0, dtype=torch.int32, device="cuda"), 1)
    assert pack.add(torch.empty(0, 20, device="cuda"), torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), empty).shape == (0, 20)


def test_infinities_stay_with_their_token():
    rng = np.random.default_rng(7)
    ads = _adapters(rng, 40, 64, [16])
    x = _bf16(rng, 3, 64)
    x[1, 5] = float("inf")
    pack = lora.LoraPack(ads)
    batch = lora.LoraBatch(torch.zeros(3, dtype=torch.int32, device="cuda"), 1)
    got = pack.add(torch.zeros(3, 40, device="cuda"), x.cuda(), batch).cpu()
    assert torch.isfinite(got[[0, 2]]).all() and not torch.isfinite(got[1]).any()


GEMM = [(64, 2048, 1), (17, 14336, 3), (163, 14336, 54), (1199, 8192, 7), (5, 20480, 64), (2500, 4096, 2), (300, 2048, 5), (33, 4096, 7), (96, 4096, 8), (200, 6144, 16), (128, 4096, 17), (64, 8192, 64),
        (1024, 2048, 64)]


@pytest.mark.parametrize("rows,cols,tokens", GEMM)
def test_product_with_adapters(rows, cols, tokens):
    print("gemm lora", rows, cols, tokens, flush=True)
    rng = np.random.default_rng(rows + cols + tokens)
    w = _bf16(rng, rows, cols, size=0.02)
    ads = _adapters(rng, rows, cols, [16, 5, 40])
    of = [int(a) for a in rng.integers(-1, 3, tokens)]
    x = _bf16(rng, tokens, cols)
    plan = codec.FixedPlan(codec.fixed_encode_device(w.cuda()))
    pack = lora.LoraPack(ads)
    batch = lora.LoraBatch(torch.tensor(of, dtype=torch.int32, device="cuda"), 3)
    x64, w64 = _f64(x), _f64(w)
    base = x64 @ w64.T
    # the batched product's own bound (cols additions, 17 more for slices and halves), then the adapters'
    own = 2 * (cols + 17) * 2.0 ** -24 * (np.abs(x64) @ np.abs(w64).T)
    ref, loose = S.lora(base, x64, of, _oracle(ads))
    a = plan.gemm_lora(x.cuda(), rows, cols, pack, batch)
    b = plan.gemm_lora(x.cuda(), rows, cols, pack, batch, out=torch.full((tokens, rows), float("nan"), device="cuda"))
    assert (plan.block_status() == 0).all()
    assert np.all(np.abs(_f64(a) - ref) <= own + loose)
    assert torch.equal(a, b)
    none = [t for t, i in enumerate(of) if i < 0]
    if cols == 2048:                # one panel, so the same sums as the product without adapters
        assert torch.equal(a[none], plan.gemm(x.cuda(), rows, cols)[none])


@pytest.mark.parametrize("rows,cols,tokens", [(4200, 6144, 20), (4100, 10240, 12), (100, 2048, 33), (3001, 2048, 20), (77, 2048, 48)])
def test_product_with_adapters_in_rounds(rows, cols, tokens):
    """More workgroups than run at once, in two or three shares; one share with X in operand order."""
    test_product_with_adapters(rows, cols, tokens)


def test_graph_replays():
    rng = np.random.default_rng(9)
    rows, cols, tokens = 256, 4096, 12
    w = _bf16(rng, rows, cols, size=0.02)
    plan = codec.FixedPlan(codec.fixed_encode_device(w.cuda()))
    pack = lora.LoraPack(_adapters(rng, rows, cols, [16, 8]))
    of = torch.tensor([0, 1] * 6, dtype=torch.int32, device="cuda")
    batch = lora.LoraBatch(of, 2)
    x = _bf16(rng, tokens, cols).cuda()
    out = torch.empty(tokens, rows, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        batch.update(of), plan.gemm_lora(x, rows, cols, pack, batch, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        batch.update(of)
        plan.gemm_lora(x, rows, cols, pack, batch, out=out)
    for k in range(4):
        x.copy_(_bf16(rng, tokens, cols))
        of.copy_(torch.from_numpy(rng.integers(-1, 2, tokens).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = lora.LoraBatch(of, 2)
        assert torch.equal(got, plan.gemm_lora(x, rows, cols, pack, eager)), k


def test_another_stream():
    rng = np.random.default_rng(10)
    pack = lora.LoraPack(_adapters(rng, 64, 96, [8]))
    x, y = _bf16(rng, 5, 96).cuda(), torch.zeros(5, 64, device="cuda")
    batch = lora.LoraBatch(torch.zeros(5, dtype=torch.int32, device="cuda"), 1)
    want = pack.add(y, x, batch, out=torch.empty_like(y))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pack.add(y, x, batch, out=torch.empty_like(y), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
