"""Low-rank adapters on the GPU with weights and tokens that are not finite."""
import numpy as np
import pytest
import torch

from lossless_entropy_coding_amd import codec, lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [4, 16, 32, 64, 128])
@pytest.mark.parametrize("cols", [1, 40, 64, 96, 200, 2048])
def test_infinite_weights_stay_infinite(rank, cols):
    """An infinity of A times a number of x is an infinity, wherever it stands
    in A: the columns past the last add nothing to it."""
    print("infinite A", rank, cols, flush=True)
    rows, tokens = 64, 5
    x = torch.ones(tokens, cols, dtype=torch.bfloat16)
    for at in sorted({0, cols // 2, cols - 1}):
        a, b = torch.full((rank, cols), 0.5, dtype=torch.bfloat16), torch.full((rows, rank), 0.25, dtype=torch.bfloat16)
        a[rank - 1, at] = float("inf")
        pack = lora.LoraPack([(a, b, 1.0), (-a, b, 2.0)])
        batch = lora.LoraBatch(torch.tensor([0, 1, -1, 0, 1], dtype=torch.int32, device="cuda"), 2)
        inf = float("inf")
        want = torch.tensor([inf, -inf, 3.0, inf, -inf], device="cuda")[:, None].expand(tokens, rows)
        for y32 in (True, False):
            y = torch.full((tokens, rows), 3.0, device="cuda", dtype=torch.float32 if y32 else torch.bfloat16)
            # (rank 16 or less: the padded ranks of B are zeros against zeros of t)
            got = pack.add(y, x.cuda(), batch)
            assert torch.equal(got.float(), want), (at, y32)
    if cols == 2048:
        plan = codec.FixedPlan(codec.fixed_encode(np.full(rows * cols, 0x3C00, np.uint16)))
        got = plan.gemm_lora(x.cuda(), rows, cols, pack, batch)
        assert torch.equal(torch.isinf(got), torch.isinf(want)) and not torch.isnan(got).any()


@pytest.mark.parametrize("rank", [1, 4, 15, 16, 17, 33, 65, 128])
def test_infinite_tokens_stay_infinite(rank):
    """An infinity of x times positive weights is one: the ranks that storage
    adds to an adapter's own add nothing.  Another adapter of the pack has the
    full rank of the storage."""
    rows, cols, inf = 64, 2048, float("inf")
    one = lambda *shape: torch.full(shape, 0.5, dtype=torch.bfloat16)   # noqa: E731
    full = next(r for r in (16, 32, 64, 128) if r >= rank)
    pack = lora.LoraPack([(one(rank, cols), one(rows, rank), 1.0), (one(full, cols), one(rows, full), -1.0)])
    of = [0, 1, -1, 0, 0, 1]
    batch = lora.LoraBatch(torch.tensor(of, dtype=torch.int32, device="cuda"), 2)
    x = torch.ones(6, cols, dtype=torch.bfloat16)
    x[0, 5], x[1, cols - 1], x[2, 0] = inf, inf, inf
    for y32 in (True, False):
        got = pack.add(torch.zeros(6, rows, device="cuda", dtype=torch.float32 if y32 else torch.bfloat16), x.cuda(), batch).float()
        assert bool((got[0] == inf).all() and (got[1] == -inf).all() and (got[2] == 0).all()) and torch.isfinite(got[3:]).all()
    plan = codec.FixedPlan(codec.fixed_encode(np.full(rows * cols, 0x3C00, np.uint16)))
    got = plan.gemm_lora(x.cuda(), rows, cols, pack, batch)
    assert bool((got[[0, 2]] == inf).all()) and torch.isnan(got[1]).all() and torch.isfinite(got[3:]).all()
