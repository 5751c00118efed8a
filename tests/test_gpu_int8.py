"""Rows in 8-bit integers and lora_linear_int8 against the 64-bit oracle.

lora_quantize_rows into int8 is exact by its definition: the scale is max|x| / 127
rounded to fp32 (one division, compared bit for bit) and the integers are those
nearest to the exact quotients, compared bit for bit.

lora_rms_norm into int8: v is off by less than UNIT = 2^-18 (test_gpu_rms_norm.py), so
an integer is off by half a step and 128 UNIT at most.

lora_linear_int8: the base sum is exact; its conversion to fp32, the scales' product
and the product with it are off by 2^-24 each, 4 x 2^-24 of the base term together;
the delta as in test_gpu_linear_fp8.py; half a bf16 step, 2^-8, of the output.  The
sums that join in fp32 (eight wavefronts' parts of K in the decode form) add
16 x 2^-24 of the magnitudes."""
import numpy as np
import pytest
import torch

from oracle import decoder as O
from oracle import experts as X
from tests import test_gpu_linear_fp8 as FP8
from tests.test_gpu_rms_norm import HALF, UNIT, draw, near

pytestmark = pytest.mark.gpu
I8 = torch.int8
F64 = lambda t: t.detach().double().cpu().numpy()     # noqa: E731


def quantize(x):
    import adapter_lora_amd as ml
    out8 = torch.full(x.shape, 99, dtype=I8, device="cuda")
    scale = torch.empty(x.shape[0], device="cuda")
    ml.lora_quantize_rows(x, out8, scale)
    return out8, scale


def check_exact(x):
    out8, scale = quantize(x)
    q, s = X.quantize_int8(F64(x.float()))
    assert np.array_equal(F64(scale), s)
    got = out8.cpu().numpy()
    bad = np.argwhere(got != q)
    assert bad.size == 0, (len(bad), bad[:4].tolist(), [(got[tuple(b)], q[tuple(b)]) for b in bad[:4]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (70, 1000), (257, 4096), (9, 8200), (6, 14336), (1, 32768)])
def test_quantize_rows_exact(M, K, dtype):
    x = draw(M, K, dtype, 4)
    x[0] = 0
    x[-1, ::3] *= 1e-3
    check_exact(x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows_ties_and_their_neighbours(dtype):
    """Values of (n + 1/2) scales and the values next to them: with a largest value of
    127 2^j the quotients are ties, with another the scale's rounding decides."""
    rows = []
    for j in range(-20, 21, 5):
        n = torch.arange(-127, 127, dtype=torch.float64) + 0.5
        rows.append(torch.cat([n * 2.0 ** j, torch.tensor([127.0 * 2.0 ** j, 0.0], dtype=torch.float64)]))
    g = torch.Generator().manual_seed(1)
    for top in (torch.rand(300, generator=g) + 1).tolist():
        t = float(torch.tensor(top).to(dtype))
        n = torch.arange(-127, 127, dtype=torch.float64) + 0.5
        near_tie = (n * (t / 127)).to(dtype).double()
        near_tie[::5] = t / 2
        rows.append(torch.cat([near_tie, torch.tensor([t, -t], dtype=torch.float64)]))
    check_exact(torch.stack(rows).to(dtype).cuda())


def test_quantize_rows_smallest_and_largest():
    """Denormal rows (the scale stays at the smallest normal number), the largest fp32."""
    x = torch.zeros(6, 16)
    x[0, :4] = torch.tensor([1e-44, -1e-44, 3e-45, 0])
    x[1, :3] = torch.tensor([1.2e-38, -6e-39, 2e-40])
    x[2, :3] = torch.tensor([1.5e-36, 7e-39, -1e-38])
    x[3, :3] = torch.tensor([3.4e38, -1.7e38, 1.33e36])
    x[4, :2] = torch.tensor([2.0 ** -119 * 127, 2.0 ** -120])
    x[5, :2] = torch.tensor([-1.0, 0.5])
    check_exact(x.cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows_infinities_and_nan(dtype):
    x = draw(5, 72, dtype, 5)
    x[0, 3], x[0, 70] = float("inf"), float("-inf")
    x[1, 5] = float("nan")
    x[2, 5], x[2, 6] = float("nan"), float("inf")
    clean = x.clone()
    clean[:3] = 1.0
    out8, scale = quantize(x)
    assert torch.isinf(scale[0]) and torch.isnan(scale[1]) and torch.isnan(scale[2])
    want = torch.zeros(72, dtype=I8, device="cuda")
    want[3], want[70] = 127, -127
    assert torch.equal(out8[0], want)
    ref8, ref = quantize(clean)
    assert torch.equal(out8[3:], ref8[3:]) and torch.equal(scale[3:], ref[3:])


def test_quantize_rows_strided():
    wide = torch.full((34, 640), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = wide[:33, 8:528]
    x.copy_(draw(33, 520, torch.bfloat16, 6))
    import adapter_lora_amd as ml
    o = torch.full((34, 560), 55, dtype=I8, device="cuda")
    scale = torch.empty(33, device="cuda")
    ml.lora_quantize_rows(x, o[:33, 16:536], scale)
    ref, s = quantize(x.contiguous())
    assert torch.equal(o[:33, 16:536], ref) and torch.equal(s, scale)
    assert (o[33] == 55).all() and (o[:, :16] == 55).all() and (o[:, 536:] == 55).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (5, 512), (33, 1032), (64, 4096), (9, 8200), (3, 16384), (1, 32768)])
def test_rms_norm_int8(M, K, dtype):
    import adapter_lora_amd as ml
    x, res = draw(M, K, dtype, 1), draw(M, K, dtype, 2, 3.0)
    w = (1 + 0.1 * draw(1, K, torch.float32, 3)[0]).to(dtype)
    out, res_out = torch.empty_like(x), torch.empty_like(x)
    out8, scale = torch.empty(M, K, dtype=I8, device="cuda"), torch.empty(M, device="cuda")
    ml.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=res_out, out=out, out8=out8, scale=scale)
    h, v = O.rms_norm(F64(x), F64(w), 1e-5, F64(res))
    near(F64(res_out), h, HALF[dtype] * 1.0001, what="residual")
    near(F64(out), v, HALF[dtype] + UNIT, what="out")
    near(F64(scale), np.abs(v).max(1) / 127, UNIT, what="scale")
    q = v / F64(scale)[:, None]
    assert (np.abs(F64(out8) - q) <= 0.5 + 128 * UNIT).all()
    # the same integers, scale and norm without the other outputs
    alone8, alone = torch.empty_like(out8), torch.empty_like(scale)
    ml.lora_rms_norm(x, w, 1e-5, residual=res, out8=alone8, scale=alone)
    assert torch.equal(alone8, out8) and torch.equal(alone, scale)


# ---------------------------------------------------------------- the projection
class Case(FP8.Case):
    def __init__(self, M, K, sizes, ranks, ids, seed=0, integers=False):
        super().__init__(M, K, sizes, ranks, ids, seed, integers)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        if integers:
            self.x8, self.W8 = self.x.to(I8), self.W8.float().to(I8)
        else:
            self.x8 = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=I8)
            self.W8 = torch.randint(-128, 128, (self.N, K), generator=g, device="cuda", dtype=I8)

    def run(self, y=None, x8=None, W8=None, x=None, stream=None):
        import adapter_lora_amd as ml
        y = torch.full((self.M, self.N), float("nan"), dtype=torch.bfloat16, device="cuda") if y is None else y
        ml.lora_linear_int8(self.table, self.W8 if W8 is None else W8, self.ws, self.x8 if x8 is None else x8,
                            self.xs, self.x if x is None else x, self.seg, y, self.ws_buf, stream=stream)
        return y

    def check(self, y):
        import adapter_lora_amd as ml
        want, mag, dmag = self.oracle()
        delta = (2 * self.K + 256) * 2.0 ** -24 + 2.0 ** -16
        got = F64(y)
        bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 20 * 2.0 ** -24 * mag + delta * dmag)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
        assert np.linalg.norm(got - want) <= 0.0025 * np.linalg.norm(want)
        assert ml.lora_read_device_error(self.ws_buf.buf) == 0


@pytest.mark.parametrize("name", list(FP8.CASES))
def test_linear_int8_matches_oracle(name):
    print(name, flush=True)
    c = Case(*FP8.CASES[name])
    c.check(c.run())


@pytest.mark.parametrize("M", [7, 40, 200])
def test_linear_int8_integers_bit_exact(M):
    c = Case(M, 64, [64, 32], [16, 32, 0], None, seed=3, integers=True)
    want = c.oracle()[0]
    got = F64(c.run())
    small = np.abs(want) <= 256
    assert small.any() and np.array_equal(got[small], want[small])


@pytest.mark.parametrize("M", [1, 30, 100, 300])
def test_linear_int8_largest_sums(M):
    """Every product 127 x 127 or (-128) x (-128), K large: sums near 2^29, all exact,
    far past what 24 bits hold."""
    K = 32768
    c = Case(M, K, [64], [0], [-1] * M, seed=2)
    c.x8.fill_(-128), c.W8.fill_(-128)
    c.x8[::2, :] = 127
    c.W8[1::2, :] = 127
    c.W8[:, 5] = 1
    c.check(c.run())


@pytest.mark.parametrize("M", [20, 100])
def test_linear_int8_strided_operands_and_neighbours(M):
    c = Case(M, 528, [120, 40], [16, 64, 0], None, seed=4)

    def wide8(t, pad):
        buf = torch.full((t.shape[0] + 1, t.shape[1] + pad), 127, dtype=I8, device="cuda")
        buf[:t.shape[0], 16:16 + t.shape[1]] = t
        return buf[:t.shape[0], 16:16 + t.shape[1]]

    xw = torch.full((M, 528 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:, 8:536] = c.x
    yw = torch.full((M + 1, 160 + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    y = c.run(y=yw[:M, 8:168], x8=wide8(c.x8, 48), W8=wide8(c.W8, 32), x=xw[:, 8:536])
    c.check(y)
    assert (yw[M] == 5).all() and (yw[:, :8] == 5).all() and (yw[:, 168:] == 5).all()


@pytest.mark.parametrize("M", [24, 150])
def test_linear_int8_repeats_bit_identical(M):
    c = Case(M, 1040, [264], [16, 32, 64], None, seed=5)
    first = c.run()
    c.check(first)
    side = torch.cuda.Stream()
    for i in range(6):
        torch.cuda.synchronize()
        again = c.run(stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


@pytest.mark.parametrize("M", [32, 200])
def test_linear_int8_graph_replays(M):
    c, d = Case(M, 512, [128], [16, 32], None, seed=7), Case(M, 512, [128], [16, 32], None, seed=8)
    y = torch.zeros(M, 128, dtype=torch.bfloat16, device="cuda")
    c.run(y)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run(y, stream=torch.cuda.current_stream())
    for i in range(5):
        src = d if i % 2 else c
        x8, xs, x = src.x8.clone(), src.xs.clone(), src.x.clone()
        c.x8.copy_(x8), c.xs.copy_(xs), c.x.copy_(x)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, c.run())
        torch.cuda.synchronize()
        c.check(got)


@pytest.mark.parametrize("M", [40, 200])
def test_norm_into_the_projection(M):
    """The norm's integers and scales, and its bf16 output beside them, into the
    projection and its adapters, as a layer runs them; against each call's own inputs."""
    import adapter_lora_amd as ml
    c = Case(M, 1040, [264, 40], [16, 64, 0], None, seed=9)
    h = draw(M, 1040, torch.bfloat16, 10, 3.0)
    w = (1 + 0.1 * draw(1, 1040, torch.float32, 11)[0]).to(torch.bfloat16)
    ml.lora_rms_norm(h, w, 1e-6, out=c.x, out8=c.x8, scale=c.xs)
    W = draw(c.N, 1040, torch.bfloat16, 12, 0.03)
    ml.lora_quantize_rows(W, c.W8, c.ws)
    c.check(c.run())


def test_nan_row_stays_in_its_row():
    c = Case(40, 512, [64], [16, 32], None, seed=6)
    clean = F64(c.run())
    c.xs[3] = float("nan")
    y = F64(c.run())
    rest = [m for m in range(40) if m != 3]
    assert np.isnan(y[3]).all() and np.array_equal(y[rest], clean[rest])
