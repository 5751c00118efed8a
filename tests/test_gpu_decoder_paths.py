"""Forms of the 8-bit decoder-layer calls that a rule on sizes chooses, each at
a size that makes it the chosen one.  Tolerances are those of the files that
Case and Layer come from."""
import numpy as np
import pytest
import torch

from oracle import decoder as O
from tests.test_gpu_linear_fp8 import E4M3, F64, Case
from tests.test_gpu_moe_decode import Layer
from tests.test_gpu_rms_norm import draw, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,sizes,L", [(260, 272, [264, 72], 48), (260, 272, [264, 72], 63), (130, 528, [40], 40),
                                         (300, 144, [13320], 50), (450, 1040, [15688, 72], 50)])
def test_infinities_of_a_late_slot_stay_with_its_tokens(M, K, sizes, L):
    """Past 64 tokens, with tables of up to 63 slots: an infinite and a NaN value
    in the B of an adapter whose slot and whose segment are 32 or more."""
    import adapter_lora_amd as ml
    g = torch.Generator().manual_seed(L)
    ids = (torch.arange(M)[torch.randperm(M, generator=g)] % (L + 1) - 1).tolist()
    c = Case(M, K, sizes, [16, 32] * (L // 2) + [64] * (L % 2), ids, seed=L)
    clean = c.run()
    c.check(clean)
    order = c.seg.req_to_lora[:int(c.seg.num_segments.item())].tolist()
    assert len(order) == L
    late = [i for i in order[32:] if i >= 32]
    i = late[-1]
    c.B[i][3, 1] = float("inf")
    c.B[i][sum(sizes) - 1, 0] = float("nan")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    y = c.run()
    other = c.ids != i
    assert torch.equal(y[other], clean[other])
    hit = [3, c.N - 1]
    assert not torch.isfinite(y[~other][:, hit]).any()
    rest = [n for n in range(c.N) if n not in hit]
    assert torch.equal(y[~other][:, rest], clean[~other][:, rest])
    assert ml.lora_read_device_error(c.ws_buf.buf) == 0


# (M, K, slices, ranks): units of 128 x 256 need four times as many small ones, and
# the longer K the fewer
LARGE = {
    "ragged": (450, 1040, [15688, 72], [20, 0, 64, 8]),
    "many_slots": (450, 1040, [15688, 72], [16, 32] * 40),
    "one_segment": (400, 1168, [16120], [64]),
    "long_k": (300, 4112, [13320], [16, 64, 0]),
}


@pytest.mark.parametrize("name", list(LARGE))
def test_large_units_match_oracle(name):
    M, K, sizes, ranks = LARGE[name]
    print(name, flush=True)
    c = Case(M, K, sizes, ranks, None, seed=len(name))
    c.check(c.run())


def test_large_units_integers_bit_exact():
    """All 32 stages of K = 4096 with factors in {-1, 0, 1}: sums are exact in
    fp32, outputs up to 256 in bf16."""
    c = Case(280, 4096, [13320], [16, 32, 0], None, seed=3, integers=True)
    want = c.oracle()[0]
    got = F64(c.run())
    small = np.abs(want) <= 256
    assert small.mean() > 0.5 and np.array_equal(got[small], want[small])


def test_large_units_adapters_infinities_stay_with_its_tokens():
    import adapter_lora_amd as ml
    c = Case(450, 1040, [15688, 72], [16, 32, 64], None, seed=5)
    clean = c.run()
    c.check(clean)
    c.B[1][3, 1] = float("inf")
    c.B[1][15687, 0] = float("nan")
    c.B[1][15700, 31] = float("-inf")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, c.sizes, c.K, torch.bfloat16)
    y = c.run()
    other, hit = c.ids != 1, [3, 15687, 15700]
    assert torch.equal(y[other], clean[other])
    assert not torch.isfinite(y[~other][:, hit]).any()
    y[:, hit] = clean[:, hit]
    assert torch.equal(y, clean)


# (M, K, slices, ranks): slice widths that cut a unit's second 16 columns, K past one
# round of a workgroup's blocks, S by way of partial sums
FORMS = {
    # decode, units of 32 columns
    "wide_one_token_three_rounds": (1, 4112, [4104, 1032, 1064], [16, 64, 32]),
    "wide_sixteen": (16, 1040, [2568, 1544], [16, 0, 64, 20]),
    "wide_nine_long_k": (9, 8208, [14344], [32, 16, 0]),
    "wide_seventeen": (17, 2064, [4104, 4104], [20, 64, 16]),
    "wide_thirty_two": (32, 528, [8216], [16, 32, 64] * 11),
    "wide_thirty_three": (33, 1040, [8216], [64, 16]),
    "wide_full": (64, 4112, [5128, 3080], [16, 0, 64, 20] * 10),
    "wide_many_slots": (64, 272, [8200], [16, 32] * 50),
    # decode, K past one round: consumers and, on halves or all of K, producers
    "long_k_one": (1, 8208, [40], [64]),
    "long_k_twenty": (20, 8208, [72], [16, 64, 0, 32]),
    "long_k_full": (64, 8208, [24, 8], [16, 32]),
    "one_chunk": (64, 2576, [264, 72, 40], [64, 16] * 20),
    "one_chunk_many_slots": (64, 2576, [72], [64, 16] * 70),
    # groups of 64 tokens, units of 32 columns
    "groups_wide": (129, 2064, [1032, 1024], [16, 64, 0]),
    "groups_wide_four": (200, 4112, [1000, 640], [20, 64]),
    "groups_wide_two_many_slots": (70, 2064, [4088], [16, 32] * 45),
    # S by way of partial sums, before each product
    "partial_sums_small_units": (700, 1040, [264, 72], [64, 16, 0, 20]),
    "partial_sums_groups": (520, 2064, [200, 56, 8], [64, 16, 0, 20]),
    "partial_sums_large_units": (450, 1040, [15640, 40, 16], [64, 16, 0, 20] * 18),
}


@pytest.mark.parametrize("name", list(FORMS))
def test_every_form_matches_oracle(name):
    M, K, sizes, ranks = FORMS[name]
    print(name, flush=True)
    c = Case(M, K, sizes, ranks, None, seed=len(name))
    y = c.run()
    c.check(y)
    torch.cuda.synchronize()
    assert torch.equal(y, c.run())


# More units (groups of an expert's tokens times 16 inner columns) than the first
# launch has consumers (768), so that each walks to other experts, rows and tokens
UNITS = {
    "few_tokens_fp8": dict(M=8, E=3, topk=2, H=48, I=6160, L=3, r=16, w8=True),
    "few_tokens": dict(M=5, E=4, topk=3, H=200, I=3208, L=2, r=48),
    "to_sixteen": dict(M=14, E=2, topk=2, H=136, I=8200, L=3, r=32),
    "to_sixteen_fp8": dict(M=16, E=2, topk=2, H=272, I=7184, L=2, r=16, w8=True, renorm=True),
    "many_experts_fp8": dict(M=27, E=12, topk=3, H=144, I=3216, L=4, r=32, w8=True),
    "some_experts": dict(M=20, E=4, topk=1, H=72, I=4104, L=3, r=16),
    "busy_experts_fp8": dict(M=40, E=4, topk=2, H=144, I=4112, L=5, r=16, w8=True),
    "two_groups_each": dict(M=64, E=4, topk=3, H=72, I=4104, L=4, r=16),
    "two_groups_each_fp8": dict(M=64, E=3, topk=2, H=80, I=4112, L=4, r=16, w8=True, renorm=True),
    "s_past_lds": dict(M=32, E=9, topk=3, H=72, I=2056, L=6, r=64),
    "s_past_lds_fp8": dict(M=48, E=9, topk=3, H=80, I=2064, L=6, r=64, w8=True),
    "s_past_lds_to_sixteen": dict(M=16, E=16, topk=8, H=72, I=1000, L=4, r=48),
    "shared_outer": dict(M=33, E=8, topk=2, H=80, I=1608, L=3, r=32, shared=True),
    "long_rows_fp8": dict(M=27, E=10, topk=4, H=2064, I=1424, L=6, r=32, w8=True, renorm=True),
}


@pytest.mark.parametrize("name", list(UNITS))
def test_moe_several_units_a_consumer(name):
    print(name, flush=True)
    layer = Layer(**UNITS[name], seed=len(name))
    out = layer.run()
    layer.check(out)
    chosen = torch.bincount(layer.topk_ids.flatten().long(), minlength=layer.E)
    groups = int(((chosen + 31) // 32).sum())
    assert groups * ((layer.I + 15) // 16) > 768
    torch.cuda.synchronize()
    assert torch.equal(out, layer.run())


@pytest.mark.parametrize("kw", [dict(M=2, E=2, topk=1, H=24592, I=40, L=2), dict(M=33, E=2, topk=1, H=16400, I=48, L=2, w8=True)])
def test_moe_one_split(kw):
    """So many output columns that one workgroup has each tile of them alone."""
    print(kw, flush=True)
    layer = Layer(**kw)
    layer.check(layer.run())


@pytest.mark.parametrize("w8", [False, True])
def test_last_expert_past_32_bit_offsets_in_each_matrix(w8):
    """Every token goes to the last expert, which starts past 2^32 bytes in W_gu
    and in W_d alike; its output has the bits of a layer that holds it alone
    (renormalized, so the routing weight is 1 in both)."""
    import adapter_lora_amd as ml
    E, H, I = 120 if w8 else 60, 4096, 9568
    small = Layer(M=5, E=1, topk=1, H=H, I=I, L=0, renorm=True, w8=w8)
    dt = torch.uint8 if w8 else torch.bfloat16
    W_gu = torch.zeros(E, 2 * I, H, dtype=dt, device="cuda")
    W_d = torch.zeros(E, H, I, dtype=dt, device="cuda")
    for big, one in ((W_gu, small.W_gu), (W_d, small.W_d)):
        big[E - 1] = one[0].view(dt)
        assert big.stride(0) * big.element_size() * (E - 1) >= 1 << 32
    s_gu = s_d = None
    if w8:
        W_gu, W_d = W_gu.view(E4M3), W_d.view(E4M3)
        s_gu, s_d = torch.zeros(E, 2 * I, device="cuda"), torch.zeros(E, H, device="cuda")
        s_gu[E - 1], s_d[E - 1] = small.s_gu[0], small.s_d[0]
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    router[:E - 1, 0] = -1000.0
    x = small.x
    x[:, 0] = 1.0
    want = small.run()
    ex = ml.MoeExperts(router, W_gu, W_d, 1, renormalize=True, s_gu=s_gu, s_d=s_d)
    ws = ml.Workspace(ml.lora_moe_decode_workspace_size(None, ex, 5))
    out = torch.empty_like(want)
    ids = torch.empty(5, 1, dtype=torch.int32, device="cuda")
    ml.lora_moe_decode(None, ex, None, x, out, ws, topk_ids=ids)
    torch.cuda.synchronize()
    assert (ids == E - 1).all() and torch.equal(out, want)
    assert out.float().abs().max() > 0


@pytest.mark.parametrize("M,K", [(1, 512), (37, 4096), (5, 14336)])
def test_norm_and_quantization_captured_and_replayed(M, K):
    """Captured once, replayed with new inputs and eager work between."""
    import adapter_lora_amd as ml
    x, res, w = (draw(m, K, torch.bfloat16, i) for i, m in enumerate((M, M, 1)))
    other = [(draw(M, K, torch.bfloat16, 10 + i), draw(M, K, torch.bfloat16, 20 + i, 3.0)) for i in range(5)]

    def outputs():
        e8 = lambda: torch.zeros(M, K, dtype=E4M3, device="cuda")     # noqa: E731
        return [torch.zeros_like(x), torch.zeros_like(x), e8(), torch.zeros(M, device="cuda"), e8(),
                torch.zeros(M, device="cuda")]

    def run(o):
        ml.lora_rms_norm(x, w[0], 1e-5, residual=res, residual_out=o[0], out=o[1], out8=o[2], scale=o[3])
        ml.lora_quantize_rows(o[1], o[4], o[5])

    got, eager = outputs(), outputs()
    run(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for a, b in other:
        x.copy_(a), res.copy_(b)
        for t in got:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        run(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(got, eager))
        assert got[1].float().abs().max() > 0


@pytest.mark.parametrize("K,lane,waves", [(64, 8, 1), (512, 8, 1), (1024, 8, 2), (4096, 8, 8), (8192, 8, 16),
                                          (16384, 16, 16), (32768, 32, 16)])
def test_norm_fp32_within_its_count_of_roundings(K, lane, waves):
    """In units of u = 2^-24: a lane adds `lane` squares one after the other, six
    additions join a wavefront's lanes and `waves` the wavefronts; with a
    square's own rounding, those of h = x + residual (once in each factor), of
    the mean and of the added eps, the sum is off by lane + waves + 11 u, its
    square root by half of that; the root, the reciprocal, the two products
    and h add one each, the stored fp32 value is the last product itself."""
    import adapter_lora_amd as ml
    x, res = draw(33, K, torch.float32, 1), draw(33, K, torch.float32, 2, 3.0)
    w = (1 + 0.1 * draw(1, K, torch.float32, 3)[0])
    out, res_out = torch.empty_like(x), torch.empty_like(x)
    ml.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=res_out, out=out)
    h, v = O.rms_norm(F64(x), F64(w), 1e-5, F64(res))
    near(F64(res_out), h, 2.0 ** -24, what="residual")
    # a sum near zero has lost nothing: it is one rounding of the exact value
    near(F64(out), v, ((lane + waves + 11) / 2 + 5) * 2.0 ** -24 * 1.001, what="out")
