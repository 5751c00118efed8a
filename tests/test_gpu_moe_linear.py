"""lora_moe_group and lora_moe_linear against the 64-bit oracle.

Groups are compared bit for bit.  Tolerance of one output of a product, as a bound:
  * half a bf16 step, 2^-8 of it;
  * bf16: fp32 sums of K exact products, (2 K + 256) 2^-24 of the sum of their
    magnitudes;
  * e4m3: as in test_gpu_linear_fp8.py, the matrix unit drops less than 7 x 2^-13 of
    the largest of every eight products, and the fp32 sum over the eights adds
    (K + 64) 2^-24 of the magnitudes;
  * int8: the sum is exact; its conversion to fp32, the scales' product and its
    own product with them are three roundings, 3 x 2^-24 of the output (4 with
    their products)."""
import numpy as np
import pytest
import torch

from oracle import experts as X

pytestmark = pytest.mark.gpu
BF, E4M3, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
TYPES = {"bf16": BF, "e4m3": E4M3, "int8": I8}
F64 = lambda t: t.detach().double().cpu().numpy()     # noqa: E731


# ---------------------------------------------------------------- groups
@pytest.mark.parametrize("M,topk,E", [(1, 1, 1), (1, 2, 8), (3, 16, 256), (31, 2, 5), (64, 1, 64), (65, 3, 63),
                                      (1000, 2, 8), (1024, 16, 129), (1025, 16, 200), (4099, 4, 65), (8191, 2, 255),
                                      (5000, 13, 7), (40000, 2, 128)])
@pytest.mark.parametrize("spread", ["even", "skewed", "one", "none", "outside"])
def test_group_bit_exact(M, topk, E, spread):
    import adapter_lora_amd as ml
    g = torch.Generator().manual_seed(M + E)
    if spread == "even":
        ids = torch.randint(0, E, (M, topk), generator=g)
    elif spread == "skewed":
        ids = (torch.rand(M, topk, generator=g) ** 4 * E).long()
    elif spread == "one":
        ids = torch.full((M, topk), E - 1)
    elif spread == "none":
        ids = torch.full((M, topk), E)
    else:
        ids = torch.randint(-3, 2 * E, (M, topk), generator=g)
        ids[::7] = -2 ** 31
    ids = ids.int()
    groups = ml.MoeGroups(M * topk + 5, E)
    groups.pairs.fill_(-9)
    ml.lora_moe_group(ids.cuda(), groups)
    pairs, offsets = X.group(ids.numpy(), E)
    assert np.array_equal(groups.pairs[:M * topk].cpu().numpy(), pairs)
    assert np.array_equal(groups.offsets.cpu().numpy(), offsets)
    assert (groups.pairs[M * topk:] == -9).all()


def test_group_no_tokens():
    import adapter_lora_amd as ml
    groups = ml.MoeGroups(4, 100)
    groups.offsets.fill_(7)
    ml.lora_moe_group(torch.empty(0, 2, dtype=torch.int32, device="cuda"), groups)
    assert not groups.offsets.any()
    y = torch.empty(0, 16, dtype=BF, device="cuda")
    ml.lora_moe_linear(torch.zeros(100, 16, 32, dtype=BF, device="cuda"),
                       torch.empty(0, 32, dtype=BF, device="cuda"), 2, groups, y)


# ---------------------------------------------------------------- products
def route(M, topk, E, counts, g):
    """topk_ids with these many pairs for each expert (in a random order), or a
    router's even choice of different experts."""
    if counts is None:
        return torch.rand(M, E, generator=g).topk(topk, 1).indices.int()
    flat = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)] + [torch.full((M * topk - sum(counts),), E)])
    return flat[torch.randperm(M * topk, generator=g)].reshape(M, topk).int()


class Case:
    def __init__(self, kind, M, topk, E, N, K, counts=None, pair_rows=False, seed=0, integers=False):
        self.kind, self.M, self.topk, self.E, self.N, self.K, self.pair_rows = kind, M, topk, E, N, K, pair_rows
        g = torch.Generator().manual_seed(seed)
        self.ids = route(M, topk, E, counts, g).cuda()
        gc = torch.Generator(device="cuda").manual_seed(seed)
        rows = M * topk if pair_rows else M

        def make(*s):
            if integers:
                return torch.randint(-1, 2, s, generator=gc, device="cuda").to(TYPES[kind])
            if kind == "int8":
                return torch.randint(-128, 128, s, generator=gc, device="cuda", dtype=I8)
            return (torch.randn(*s, generator=gc, device="cuda") * (60 if kind == "e4m3" else 1)).to(TYPES[kind])

        self.x, self.W = make(rows, K), make(E, N, K)
        self.xs = self.ws = None
        if kind != "bf16":
            self.xs = torch.rand(rows, generator=gc, device="cuda") * 0.02 + 0.01
            self.ws = torch.rand(E, N, generator=gc, device="cuda") * 0.01 + 1e-3
            if integers:
                self.xs.fill_(1), self.ws.fill_(1)
        import adapter_lora_amd as ml
        self.groups = ml.MoeGroups(M * topk, E)

    def run(self, y=None, x=None, stream=None, group=True):
        import adapter_lora_amd as ml
        y = torch.full((self.M * self.topk, self.N), 77.0, dtype=BF, device="cuda") if y is None else y
        if group:
            ml.lora_moe_group(self.ids, self.groups, stream=stream)
        ml.lora_moe_linear(self.W, self.x if x is None else x, self.topk, self.groups, y, w_scale=self.ws,
                           x_scale=self.xs, stream=stream)
        return y

    def oracle(self):
        f = lambda t: None if t is None else F64(t.float())       # noqa: E731
        return X.grouped_linear_mag(self.ids.cpu().numpy(), f(self.x), f(self.W), self.pair_rows, f(self.xs), f(self.ws))

    def check(self, y, untouched=77.0):
        want, mag = self.oracle()
        got = F64(y.float())
        on = ~np.isnan(want[:, 0])
        assert (got[~on] == untouched).all()
        got, want, mag = got[on], want[on], mag[on]
        if self.kind == "bf16":
            bound = 2.0 ** -8 * np.abs(want) + (2 * self.K + 256) * 2.0 ** -24 * mag
        elif self.kind == "e4m3":
            bound = 2.0 ** -8 * np.abs(want) + ((self.K + 64) * 2.0 ** -24 + 7 * 2.0 ** -13) * mag
        else:
            bound = (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(want)
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
        if want.size > 1000:
            assert np.linalg.norm(got - want) <= 0.0025 * np.linalg.norm(want)


# (M, topk, E, N, K, pairs of each expert, rows of x per pair)
CASES = {
    "one_pair": (1, 1, 1, 8, 16, None, False),
    "one_token": (1, 2, 8, 264, 528, None, False),
    "one_token_short_k": (1, 4, 40, 72, 16, None, True),
    "few": (9, 2, 8, 1000, 1040, None, False),
    "few_busy_expert": (30, 2, 20, 136, 272, [0, 45, 1, 0, 3, 1], False),
    "few_16_rows": (16, 4, 4, 40, 2064, [16, 16, 16, 16], True),
    "few_33_rows": (33, 2, 8, 24, 144, [33, 0, 1], False),
    "same_expert_twice": (12, 4, 3, 48, 96, [20, 0, 28], False),
    "tile_64": (64, 2, 2, 264, 1040, [64, 64], False),
    "tile_65": (65, 2, 2, 256, 256, [65, 64], True),
    "tile_ragged": (700, 2, 6, 272, 400, [1, 128, 129, 192, 193, 256], False),
    "tile_257_rows": (300, 2, 3, 520, 80, [257, 0, 343], True),
    "tile_bands": (1500, 1, 2, 24, 48, [1400, 90], False),
    "tile_one_k_chunk": (300, 1, 2, 64, 16, None, False),
    "tile_two_stages": (300, 1, 2, 64, 256, None, True),
    "tile_three_stages": (300, 1, 2, 64, 288, None, False),
    "tile_four_stages": (310, 1, 2, 64, 400, None, True),
    "tile_long_k": (260, 1, 1, 16, 8208, None, False),
    "many_experts": (2000, 3, 256, 32, 64, None, False),
    "rows_elsewhere": (900, 2, 5, 136, 144, [300, 0, 20, 200, 1], False),
    "nothing_here": (40, 2, 3, 16, 32, [0, 0, 0], False),
    "wide": (70, 2, 2, 2312, 128, None, True),
    "tiles_in_order": (600, 2, 6, 20008, 16, [300, 64, 0, 200, 513, 90], False),
    "tiles_in_order_many_experts": (1500, 2, 130, 1096, 32, None, False),
    "few_256_experts": (500, 4, 256, 40, 48, None, True),
    "few_32_rows": (64, 2, 8, 24, 272, [30, 2, 33, 1, 31, 0, 16, 15], False),
    "few_one_expert_of_many": (300, 1, 200, 72, 160, [0] * 150 + [300], False),
    # tiles of all 256 columns: 256 and more of them
    "whole_tiles": (3000, 2, 40, 1800, 272, [1, 64, 65, 128, 129, 192, 193, 256, 257, 513, 0, 700], False),
    "whole_tiles_short_k": (1200, 4, 64, 1032, 32, None, True),
    "whole_tiles_long_k": (640, 2, 8, 8200, 2064, None, False),
    "whole_tiles_few_rows": (40, 8, 130, 520, 144, None, False),
    # starts of K that differ
    "few_parts": (130, 1, 40, 72, 160, [65, 1, 64], False),
    "few_parts_of_200": (200, 2, 200, 40, 48, [0] * 60 + [129, 0, 64] + [0] * 120 + [200, 5], True),
    "few_of_256": (60, 4, 256, 40, 48, None, True),
    "few_wide": (6, 2, 5, 2600, 4112, None, False),
    "few_wide_32_rows": (30, 2, 4, 1600, 8208, None, True),
    "few_wide_odd_steps": (4, 4, 16, 4104, 1552, None, False),
    "half_tiles_wide": (250, 2, 3, 5000, 1424, [400, 3, 97], False),
    # rows of W of whole cache lines, shares of one tile (W not kept) and of more
    "few_lines": (6, 2, 5, 600, 1152, None, False),
    "few_lines_32_rows": (30, 2, 4, 600, 640, [20, 33, 1], True),
    "half_tiles_lines": (500, 2, 4, 648, 512, [64, 128, 192, 300], False),
    "whole_tiles_lines": (700, 4, 40, 1800, 384, [60, 100, 192, 256, 257, 513], False),
}
WHOLE_TILES = [k for k in CASES if k.startswith("whole")]
FEW = [k for k in CASES if k.startswith("few") and k != "few_256_experts"]


def form(kind, P, E, N, K):
    """The form that the size rule takes."""
    Kb, shares, cols = K * (2 if kind == "bf16" else 1), min(E, P), -(-N // 256)
    if P <= 8 * shares and (Kb >= 4096 or P < 2 * E or shares * cols < 256):
        return "few"
    if P <= 16 * shares and (shares * cols < 128 or shares * cols < 256 and Kb <= 8192):
        return "few"
    return "half tiles" if (P // 256 + shares) * cols < 256 else "whole tiles"


@pytest.mark.parametrize("kind", list(TYPES))
def test_cases_reach_every_form(kind):
    def forms(names):
        return {form(kind, c[0] * c[1], *c[2:5]) for c in (CASES[k] for k in names)}
    assert forms(WHOLE_TILES) == {"whole tiles"} and forms(FEW) == {"few"}
    assert forms(["tile_ragged", "tile_long_k", "tile_257_rows", "half_tiles_wide"]) == {"half tiles"}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_moe_linear_matches_oracle(name, kind):
    print(name, kind, flush=True)
    M, topk, E, N, K, counts, pair_rows = CASES[name]
    c = Case(kind, M, topk, E, N, K, counts, pair_rows, seed=len(name))
    c.check(c.run())


@pytest.mark.parametrize("M", [3, 40, 600])
def test_bf16_k_of_eight(M):
    """bf16 rows of any multiple of 8 values: the last 16 bytes alone in their segment."""
    for K in (8, 24, 72, 200):
        c = Case("bf16", M, 2, 4, 40, K, seed=K)
        c.check(c.run())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M", [5, 90, 700])
def test_integers_bit_exact(kind, M):
    c = Case(kind, M, 2, 3, 72, 160, seed=3, integers=True)
    want = c.oracle()[0]
    got = F64(c.run().float())
    small = np.abs(want) <= 256
    assert small.all() and np.array_equal(got, want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M", [7, 500])
def test_strided_operands_and_neighbours(kind, M):
    """x and y inside wider buffers whose padding is NaN (or the largest integer) or
    a sentinel: neither is read into a result nor written."""
    c = Case(kind, M, 2, 4, 136, 336, seed=4)
    xw = torch.full((M + 1, 336 + 64), 127 if kind == "int8" else float("nan"), device="cuda").to(TYPES[kind])
    xw[:M, 16:352] = c.x
    yw = torch.full((2 * M + 1, 136 + 24), 5.0, dtype=BF, device="cuda")
    y = c.run(y=yw[:2 * M, 8:144], x=xw[:M, 16:352])
    c.check(y)
    assert (yw[2 * M] == 5).all() and (yw[:, :8] == 5).all() and (yw[:, 144:] == 5).all()


@pytest.mark.parametrize("M", [6, 400])
def test_infinities_past_k_and_in_rows(M):
    """A short last segment of K after segments with infinities: what the ring held
    before does not come back, and a row's or a column's infinity stays its own."""
    K = 64 * 5 + 8
    c = Case("bf16", M, 2, 2, 72, K, seed=5)
    c.x[2, 3], c.x[2, K - 1] = float("inf"), float("inf")
    c.W[1, 5, 64 * 3 + 9] = float("inf")
    c.x[c.x.abs() < 2 ** -6] = 1.0                               # no zero meets an infinity
    c.W[c.W.abs() < 2 ** -6] = 1.0
    want = c.oracle()[0]
    got = F64(c.run().float())
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    on = np.isfinite(want)
    assert (~on).any() and np.allclose(got[on], want[on], rtol=2 ** -7, atol=0.05)


def test_nan_scale_and_nan_value_stay_in_their_rows():
    for kind, M in (("e4m3", 6), ("e4m3", 300), ("int8", 6), ("int8", 300)):
        c = Case(kind, M, 2, 2, 40, 272, seed=6)
        clean = F64(c.run().float())
        c.xs[3] = float("nan")
        if kind == "e4m3":
            c.x.view(torch.uint8)[4, 271] = 0x7f
        y = F64(c.run().float())
        hit = [3, 4] if kind == "e4m3" else [3]
        rows = np.isin(np.arange(2 * M) // 2, hit)
        assert np.isnan(y[rows]).all() and np.array_equal(y[~rows], clean[~rows])


@pytest.mark.parametrize("kind,M", [("bf16", 10), ("int8", 300), ("e4m3", 777)])
def test_repeats_bit_identical_on_two_streams(kind, M):
    c = Case(kind, M, 2, 4, 264, 528, seed=7)
    first = c.run()
    c.check(first)
    side = torch.cuda.Stream()
    for i in range(6):
        torch.cuda.synchronize()
        again = c.run(stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


@pytest.mark.parametrize("kind,M", [("bf16", 5), ("int8", 40), ("e4m3", 600)])
def test_graph_replays(kind, M):
    """Grouping and product captured once, replayed with other tokens and experts,
    with eager work between."""
    c, d = Case(kind, M, 2, 4, 72, 272, seed=8), Case(kind, M, 2, 4, 72, 272, seed=9)
    y = torch.zeros(2 * M, 72, dtype=BF, device="cuda")
    c.run(y)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run(y, stream=torch.cuda.current_stream())
    other = Case(kind, M, 2, 4, 72, 272, seed=10)
    for i in range(6):
        src = (c, d, other)[i % 3]
        ids, x = src.ids.clone(), src.x.clone()
        c.ids.copy_(ids), c.x.copy_(x)
        y.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, c.run())
        torch.cuda.synchronize()
        c.check(got)


@pytest.mark.parametrize("kind,M", [("bf16", 4), ("e4m3", 4), ("int8", 300)])
def test_last_expert_past_32_bit_offsets(kind, M):
    """Weights of more than 4 GiB: the experts past 2^32 bytes are the ones used."""
    K, N, E = 16384, 16384 if kind == "bf16" else 32768, 9
    W = torch.zeros(E, N, K, dtype=torch.int8 if kind == "int8" else TYPES[kind], device="cuda")
    c = Case(kind, M, 1, 1, 48, K, seed=11)
    W[E - 1, N - 48:] = c.W[0]
    import adapter_lora_amd as ml
    groups = ml.MoeGroups(M, E)
    ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
    ml.lora_moe_group(ids, groups)
    y = torch.full((M, N), 3.0, dtype=BF, device="cuda")
    ws = None
    if c.ws is not None:
        ws = torch.ones(E, N, device="cuda")
        ws[E - 1, N - 48:] = c.ws[0]
    ml.lora_moe_linear(W, c.x, 1, groups, y, w_scale=ws, x_scale=c.xs)
    assert not y[:, :N - 48].any()
    c.check(y[:, N - 48:])


def test_rows_past_32_bit_offsets():
    """x and y rows whose distance from the first passes 2^32 bytes."""
    import adapter_lora_amd as ml
    for M, ld in ((9, 1 << 28), (300, 1 << 24)):
        c = Case("bf16", M, 1, 2, 72, 136, seed=12)
        flat = torch.zeros((M - 1) * ld + 136, dtype=BF, device="cuda")
        x = flat.as_strided((M, 136), (ld, 1))
        x.copy_(c.x)
        out = torch.zeros((M - 1) * ld + 72, dtype=BF, device="cuda")
        y = out.as_strided((M, 72), (ld, 1))
        ml.lora_moe_group(c.ids, c.groups)
        ml.lora_moe_linear(c.W, x, 1, c.groups, y)
        c.check(y)
        del flat, out, x, y


def test_groups_that_name_no_pair():
    """pairs and offsets from elsewhere: no row outside the batch is read or written."""
    import adapter_lora_amd as ml
    for M in (6, 400):
        c = Case("bf16", M, 2, 3, 40, 72, seed=13)
        c.run()
        yw = torch.full((2 * M + 64, 40), 5.0, dtype=BF, device="cuda")
        c.groups.pairs.fill_(2 ** 31 - 1)
        c.groups.offsets.copy_(torch.tensor([-5, 3, 2 ** 30, 7], dtype=torch.int32))
        ml.lora_moe_linear(c.W, c.x, 2, c.groups, yw[:2 * M])
        torch.cuda.synchronize()
        assert (yw[:2 * M - 1] == 5).all() and (yw[2 * M:] == 5).all()


def test_two_streams_at_once():
    """Two batches on two streams over the same weights at the same time."""
    c, d = Case("bf16", 500, 2, 4, 264, 1040, seed=14), Case("bf16", 500, 2, 4, 264, 1040, seed=15)
    d.W = c.W
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = c.run().clone(), d.run().clone()
    ys = [torch.empty_like(want[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        c.run(ys[0], stream=a)
        d.run(ys[1], stream=b)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


# ---------------------------------------------------------------- a whole layer
@pytest.mark.parametrize("kind,M", [("bf16", 6), ("bf16", 150), ("int8", 150), ("e4m3", 150)])
def test_layer_of_many_tokens(kind, M):
    """The MoE layer as a batch runs it: groups, gate/up products, deltas, activation,
    down products, deltas, reduce; each step's input is the step's before it, as
    the kernels left it."""
    import adapter_lora_amd as ml
    H, I, E, topk, L, r = 256, 160, 4, 2, 3, 16
    g = torch.Generator(device="cuda").manual_seed(16)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()    # noqa: E731
    x, ids = rnd(M, H), torch.randint(-1, L, (M,), generator=g, device="cuda").int()
    tk = torch.rand(M, E, generator=g, device="cuda").topk(topk, 1).indices.int().contiguous()
    tw = torch.rand(M, topk, generator=g, device="cuda")
    W = [rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5)]
    A = rnd(L, E, r, H, std=0.05), rnd(L, E, 2 * I, r, std=0.3), rnd(L, E, r, I, std=0.05), rnd(L, E, H, r, std=0.3)
    w = ml.MoeWeights(*A, torch.ones(L, dtype=torch.int32, device="cuda"))
    cap = ml.lora_moe_align_capacity(M, topk, E, 16)
    al = ml.MoeAlign(L, cap, 16)
    ws = ml.Workspace(ml.lora_moe_workspace_size(w, cap))
    groups = ml.MoeGroups(M * topk, E)
    new = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")       # noqa: E731
    c1, c2, c3, out = new(M * topk, 2 * I), new(M * topk, I), new(M * topk, H), new(M, H)

    def eight(t):
        rows = t.reshape(-1, t.shape[-1])
        q, s = new(*rows.shape, dtype=TYPES[kind]), new(rows.shape[0], dtype=torch.float32)
        ml.lora_quantize_rows(rows, q, s)
        return q.view(t.shape), s.view(t.shape[:-1])

    def product(Wm, rows, y):
        if kind == "bf16":
            ml.lora_moe_linear(Wm, rows, topk, groups, y)
            return
        (W8, sw), (x8, sx) = eight(Wm), eight(rows)
        ml.lora_moe_linear(W8, x8, topk, groups, y, w_scale=sw, x_scale=sx)

    ml.lora_moe_align(tk, ids, w.enabled, E, al)
    ml.lora_moe_group(tk, groups)
    product(W[0], x, c1)
    ml.lora_moe_gate_up_add(w, x, topk, al, c1, ws)
    ml.lora_moe_silu_and_mul(c1, c2)
    product(W[1], c2, c3)
    ml.lora_moe_down_add(w, c2, M, topk, al, c3, ws)
    ml.lora_moe_topk_reduce(c3, tw, out)
    # in 64 bits, pair by pair; each cache is rounded to bf16 twice and the rows and
    # weights of the 8-bit forms to 2^-4 (e4m3) or 2^-8 of the largest
    want = np.zeros((M, H))
    xd, Wg, Wd, Ad = F64(x), F64(W[0]), F64(W[1]), [F64(a) for a in A]
    for m in range(M):
        for k in range(topk):
            e, l = int(tk[m, k]), int(ids[m])
            G, D = Wg[e], Wd[e]
            if l >= 0:
                G, D = G + Ad[1][l, e] @ Ad[0][l, e], D + Ad[3][l, e] @ Ad[2][l, e]
            gu = G @ xd[m]
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            want[m] += float(tw[m, k]) * (D @ h)
    err = np.linalg.norm(F64(out) - want) / np.linalg.norm(want)
    # random roundings: bf16 caches 6 of 2^-9 / sqrt(3) at most add up to 0.01; int8 rows
    # of 256 normal values have steps of max / 127 = 3 sigma / 127, e4m3 values 2^-5 at random
    assert err <= {"bf16": 0.01, "int8": 0.04, "e4m3": 0.12}[kind], err
