"""lora_rms_norm and lora_quantize_rows against the 64-bit oracle.

Tolerances: an output in bf16 is off by half a step, 2^-8 relative, fp32
2^-24; e4m3 by 2^-4 relative above its smallest normal value 2^-6 and by half
a step of 2^-10 below.  What is computed before that rounding (a sum of K
squares in fp32, a square root, four products) is off by less than UNIT =
2^-18: the longest chain of additions in one sum is K / 64 <= 512 terms of a
lane and the joins, 64 of which, all off the same way, make 2^-18."""
import numpy as np
import pytest
import torch

from oracle import decoder as O

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F64 = lambda t: t.detach().double().cpu().numpy()     # noqa: E731


def draw(M, K, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, generator=g, device="cuda") * std).to(dtype)


def near(got, want, rel, floor=0.0, what=""):
    bad = np.abs(got - want) > rel * np.abs(want) + floor
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want).max()))


def check_eight(out8, scale, v, what):
    s = O.row_scale(v)
    near(F64(scale), s, UNIT, what=what + " scale")
    # against the scale that was stored: the value a reader reconstructs
    q = v / F64(scale)[:, None]
    got = F64(out8.float())
    assert (np.abs(got) <= 448).all()
    bad = np.abs(got - q) > np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10) + UNIT * np.abs(q)
    assert not bad.any(), (what, int(bad.sum()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (5, 512), (2, 520), (33, 1032), (7, 2056),
                                 (64, 4096), (130, 4104), (9, 8200), (3, 16384), (2, 24576),
                                 (1, 32768)])
def test_rms_norm_matches_oracle(M, K, dtype):
    import adapter_lora_amd as ml
    x, res = draw(M, K, dtype, 1), draw(M, K, dtype, 2, 3.0)
    w = (1 + 0.1 * draw(1, K, torch.float32, 3)[0]).to(dtype)
    out, res_out = torch.empty_like(x), torch.empty_like(x)
    out8 = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(M, device="cuda")
    ml.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=res_out, out=out, out8=out8,
                     scale=scale)
    h, v = O.rms_norm(F64(x), F64(w), 1e-5, F64(res))
    near(F64(res_out), h, HALF[dtype] * 1.0001, what="residual")
    near(F64(out), v, HALF[dtype] + UNIT, what="out")
    check_eight(out8, scale, v, "with residual")
    # each output alone, without a residual
    h, v = O.rms_norm(F64(x), F64(w), 1e-5)
    only, alone8, alone = torch.empty_like(x), torch.empty_like(out8), torch.empty_like(scale)
    ml.lora_rms_norm(x, w, 1e-5, out=only)
    ml.lora_rms_norm(x, w, 1e-5, out8=alone8, scale=alone)
    near(F64(only), v, HALF[dtype] + UNIT, what="out alone")
    check_eight(alone8, alone, v, "alone")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (70, 1000), (257, 4096), (6, 14336), (1, 32768)])
def test_quantize_rows_matches_oracle(M, K, dtype):
    import adapter_lora_amd as ml
    x = draw(M, K, dtype, 4)
    x[0] = 0
    x[-1, ::3] *= 1e-3
    out8 = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(M, device="cuda")
    ml.lora_quantize_rows(x, out8, scale)
    if M > 1:
        assert scale[0].item() == 1.0 and not F64(out8.float())[0].any()
    check_eight(out8, scale, F64(x), "rows")


def test_rounds_to_nearest_even_and_keeps_representable_values():
    """With the row's largest value at 448 the scale is 1: representable
    values come back exactly, and ties go to the even neighbour."""
    import adapter_lora_amd as ml
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)]                       # 254 values, 448 among them
    ties = torch.tensor([17.0, 19.0, -17.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -0.0])
    row = torch.cat([every, ties])
    x = torch.zeros(1, 264)
    x[0, :row.numel()] = row
    want = x.clone()
    want[0, 254:262] = torch.tensor([16.0, 20.0, -16.0, 1.0, 1.25, 0.0, 2.0 ** -8, -0.0])
    out8 = torch.empty(1, 264, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(1, device="cuda")
    ml.lora_quantize_rows(x.cuda(), out8, scale)
    assert scale.item() == 1.0
    assert torch.equal(out8.float().cpu(), want)


def test_extreme_rows():
    """Tiny and huge rows, NaN and infinities stay in their own rows."""
    import adapter_lora_amd as ml
    K = 1024
    x = draw(8, K, torch.float32, 5)
    x[1] *= 1e-42                                             # subnormal values
    x[2] *= 1e37
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    x[5] = 0
    out8 = torch.empty(8, K, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(8, device="cuda")
    ml.lora_quantize_rows(x, out8, scale)
    s, q = scale.cpu(), out8.float().cpu()
    assert s[1] >= 2.0 ** -126 and torch.isfinite(q[1]).all()
    assert torch.isnan(s[3]) and torch.isnan(q[3]).all()
    assert torch.isinf(s[4]) and torch.isnan(q[4, 7]) and not q[4, :7].any()
    assert s[5] == 1
    ok = [0, 2, 6, 7]
    check_eight(out8[ok], scale[ok], F64(x)[ok], "other rows")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_in_place_and_untouched_neighbours(dtype):
    import adapter_lora_amd as ml
    M, K, pad = 37, 1000, 16
    wide = torch.full((M + 1, K + pad), 7.0, dtype=dtype, device="cuda")
    x = wide[:M, 8:8 + K]
    x.copy_(draw(M, K, dtype, 6))
    res = draw(M, K, dtype, 7)
    w = draw(1, K, dtype, 8)[0]
    h, v = O.rms_norm(F64(x), F64(w), 1e-6, F64(res))
    out8w = torch.zeros(M + 1, K + 24, dtype=torch.uint8, device="cuda")
    out8 = out8w.view(torch.float8_e4m3fn)[:M, :K]
    scale = torch.full((M + 1,), -1.0, device="cuda")
    ml.lora_rms_norm(x, w, 1e-6, residual=res, residual_out=res, out=x, out8=out8,
                     scale=scale[:M])
    near(F64(res), h, HALF[dtype] * 1.0001, what="residual in place")
    near(F64(x), v, HALF[dtype] + UNIT, what="out in place")
    check_eight(out8, scale[:M], v, "strided")
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + K:] == 7).all() and (wide[M] == 7).all()
    assert not out8w[M].any() and not out8w[:, K:].any() and scale[M] == -1
    # x itself as residual_out
    y = draw(5, K, dtype, 9)
    r2 = draw(5, K, dtype, 10)
    h, v = O.rms_norm(F64(y), F64(w), 1e-6, F64(r2))
    o = torch.empty_like(y)
    ml.lora_rms_norm(y, w, 1e-6, residual=r2, residual_out=y, out=o)
    near(F64(y), h, HALF[dtype] * 1.0001)
    near(F64(o), v, HALF[dtype] + UNIT)


def test_no_rows_and_other_streams():
    import adapter_lora_amd as ml
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    ml.lora_rms_norm(e, w, out=torch.empty_like(e))
    ml.lora_quantize_rows(e, torch.empty(0, 64, dtype=torch.float8_e4m3fn, device="cuda"),
                          torch.empty(0, device="cuda"))
    x = draw(300, 64, torch.bfloat16, 11)
    a, b = torch.empty_like(x), torch.empty_like(x)
    ml.lora_rms_norm(x, w, out=a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ml.lora_rms_norm(x, w, out=b, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_more_rows_than_one_grid_axis_holds():
    """2^26 + 3 rows of eight values: more than 2^32 threads."""
    import adapter_lora_amd as ml
    M = (1 << 26) + 3
    x = torch.full((M, 8), 2.0, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 5, (1 << 23) + 1, 1 << 25, (1 << 26) - 1, 1 << 26, M - 1], device="cuda")
    x[at] = draw(len(at), 8, torch.bfloat16, 1)
    out8 = torch.zeros(M, 8, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.zeros(M, device="cuda")
    ml.lora_quantize_rows(x, out8, scale)
    check_eight(out8[at], scale[at], F64(x[at]), "rows past 2^32 threads")
    scale[at] = 2.0 / 448
    assert float((scale - 2.0 / 448).abs().max()) <= 2.0 ** -24 * 2 / 448
