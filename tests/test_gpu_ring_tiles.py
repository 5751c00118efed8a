"""The 8-bit projections in tiles of 256 x 256 (gemm_ring.hpp) at the sizes where the
size rule takes them: short and ragged last row tiles, several slices, one adapter
and many, no adapter, rows and K that end inside a tile or a stage, B with
infinities.  Tolerances are those of test_gpu_linear_fp8.py and test_gpu_int8.py."""
import numpy as np
import pytest
import torch

from tests import test_gpu_int8 as I8
from tests import test_gpu_linear_fp8 as FP8

pytestmark = pytest.mark.gpu
KINDS = {"int8": I8.Case, "e4m3": FP8.Case}

# M, K, slice sizes, ranks, ids
CASES = {
    "one_round": (512, 1024, [28672], [16, 64, 0, 32], None),
    "short_last_rows": (300, 4112, [28672], [20, 0, 64, 8], None),
    "rows_past_128": (460, 1040, [26000, 2600], [64], None),
    "three_slices": (500, 1296, [20000, 264, 8400], [16, 32], None),
    "no_adapter": (512, 1056, [28672], [16], [-1] * 512),
    "one_adapter": (512, 1168, [28672], [64], [0] * 512),
    "many_slots": (512, 1040, [28672], [16, 32] * 40, None),
    "two_rounds": (700, 1040, [43016], [32, 16, 48], None),
}


def takes_tiles(M, K, sizes):
    """The size rule of the larger 8-bit product, in its own units of time."""
    def cost(rows, width, fixed, per_k):
        units = -(-M // rows) * sum(-(-n // width) for n in sizes)
        return -(-units // 256) * (fixed * 4096 + per_k * K)
    return cost(256, 256, 130, 330) < min(cost(64, 128, 14, 85), cost(128, 256, 80, 200))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("name", list(CASES))
def test_ring_tiles_match_oracle(name, kind):
    print(name, kind, flush=True)
    assert takes_tiles(*CASES[name][:3])
    c = KINDS[kind](*CASES[name], seed=len(name))
    y = c.run()
    c.check(y)


@pytest.mark.parametrize("kind", list(KINDS))
def test_ring_tiles_infinities_stay_with_their_tokens(kind):
    """An infinity in one adapter's B: its own tokens' outputs in that column are
    infinite or NaN, all others the same bits as without it."""
    c = KINDS[kind](512, 1024, [28672], [16, 64, 32], None, seed=3)
    clean = c.run()
    c.B[1][5, 3] = float("inf")
    c.B[1][28671, 60] = float("nan")
    import adapter_lora_amd as ml
    c.table = ml.LoraTable(c.A, c.B, c.ranks, c.sizes, c.K, torch.bfloat16)
    y = c.run()
    mine = (c.ids == 1)
    assert mine.any() and (~mine).any()
    bad = ~torch.isfinite(y.float())
    assert bad[mine][:, 5].all() and bad[mine][:, 28671].all()
    bad[:, 5] &= ~mine
    bad[:, 28671] &= ~mine
    assert not bad.any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[mine, 5] = False
    keep[mine, 28671] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("kind", list(KINDS))
def test_ring_tiles_strided(kind):
    """x8, W8 and y inside wider buffers: neighbours are neither read into a result nor
    written."""
    M, K, N = 400, 1040, 28672
    assert takes_tiles(M, K, [N]) and takes_tiles(512, 1024, [N])
    c = KINDS[kind](M, K, [N], [16, 0, 32], None, seed=5)
    want = c.run()
    pad = 0x7f

    def wide8(t, extra):
        buf = torch.full((t.shape[0] + 1, t.shape[1] + extra), pad, dtype=torch.uint8, device="cuda")
        buf[:t.shape[0], 16:16 + t.shape[1]] = t.view(torch.uint8)
        return buf.view(t.dtype)[:t.shape[0], 16:16 + t.shape[1]]

    yw = torch.full((M + 1, N + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    y = c.run(y=yw[:M, 8:8 + N], x8=wide8(c.x8, 48), W8=wide8(c.W8, 32))
    assert torch.equal(y, want)
    assert (yw[M] == 5).all() and (yw[:, :8] == 5).all() and (yw[:, 8 + N:] == 5).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_ring_tiles_graph_and_streams(kind):
    c, d = (KINDS[kind](512, 1024, [28672], [16, 32], None, seed=s) for s in (7, 8))
    y = torch.zeros(512, 28672, dtype=torch.bfloat16, device="cuda")
    c.run(y)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run(y, stream=torch.cuda.current_stream())
    for i in range(4):
        src = d if i % 2 else c
        x8, xs, x = src.x8.clone(), src.xs.clone(), src.x.clone()
        c.x8.copy_(x8), c.xs.copy_(xs), c.x.copy_(x)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, c.run())
        torch.cuda.synchronize()
    assert np.isfinite(got.float().cpu().numpy()).all()
