"""Products of 8-bit integers and of experts for any number of tokens: what is measured.

Three operators that stand beside the adapters' own:

  * ``experts``: the pairs (token, chosen expert) of a batch brought into the
    experts' order, and one matrix product with each expert's weights over its
    own, ragged share of the rows, y[f] = W[e_f] x[f]: the base products that
    the MoE deltas are added to, in bf16, in e4m3 or in 8-bit integers;
  * ``linear``: a shared projection held in 8-bit integers beside the adapters of
    many requests, y = (x8 W8^T) xs ws + (x A_i^T) B_i^T, from one token to prefill;
  * ``quantize``: rows in 8-bit integers with one scale each, activations and
    weights.

Sizes: the repository's decode, prefill, stacked and MoE workloads (hidden size
4096, outputs 4096, [4096, 1024, 1024] and [14336, 14336], 8 experts of 14336,
top-2) and generic ones.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
INT8_MAX = 127.0
RANKS = (16, 32, 64, 8, 20, 0)      # adapter ranks, in turn (0: an empty slot)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token through the gate/up halves of 4 of 40 small experts: latency counts
        {"name": "experts_1_int8", "op": "experts", "M": 1, "E": 40, "topk": 4, "K": 2064, "N": 2848, "dtype": "int8", "pair_rows": False,
         "skew": 0.5},
        # 64 decoding requests through the down projections of 8 large experts
        {"name": "experts_64_down_fp8", "op": "experts", "M": 64, "E": 8, "topk": 2, "K": 14336, "N": 4096, "dtype": "e4m3", "pair_rows": True,
         "skew": 0.3},
        # a mixed batch over the gate/up halves of 8 large experts
        {"name": "experts_256_gate_up", "op": "experts", "M": 256, "E": 8, "topk": 2, "K": 4096, "N": 28672, "dtype": "bf16", "pair_rows": False,
         "skew": 0.3},
        # an odd batch over many small experts, some with most of the tokens, some with none
        {"name": "experts_1531_ragged_int8", "op": "experts", "M": 1531, "E": 64, "topk": 6, "K": 2048, "N": 2816, "dtype": "int8",
         "pair_rows": False, "skew": 1.0},
        # a prefill batch through the gate/up halves in 8 bits
        {"name": "experts_2048_gate_up_fp8", "op": "experts", "M": 2048, "E": 8, "topk": 2, "K": 4096, "N": 28672, "dtype": "e4m3",
         "pair_rows": False, "skew": 0.3},
        # a large prefill batch through the down projections
        {"name": "experts_4096_down", "op": "experts", "M": 4096, "E": 8, "topk": 2, "K": 14336, "N": 4096, "dtype": "bf16", "pair_rows": True,
         "skew": 0.3},
        # one token through the stacked query/key/value projection
        {"name": "linear_1_qkv_int8", "op": "linear", "M": 1, "K": 4096, "n0": 4096, "n1": 1024, "n2": 1024, "L": 32, "runs": 0},
        # 32 decoding requests, each with an adapter of its own choice
        {"name": "linear_32_int8", "op": "linear", "M": 32, "K": 4096, "n0": 4096, "n1": 0, "n2": 0, "L": 32, "runs": 0},
        # a mixed batch of 512 tokens through the stacked gate/up projection
        {"name": "linear_512_gate_up_int8", "op": "linear", "M": 512, "K": 4096, "n0": 14336, "n1": 14336, "n2": 0, "L": 12, "runs": 36},
        # a large prefill batch, one adapter per sequence
        {"name": "linear_8192_int8", "op": "linear", "M": 8192, "K": 4096, "n0": 4096, "n1": 0, "n2": 0, "L": 8, "runs": 11},
        # the activations before the down projection of 64 tokens
        {"name": "quantize_act_64_int8", "op": "quantize", "M": 64, "K": 14336, "dtype": "bf16"},
        # a gate/up weight brought to 8-bit integers at load time
        {"name": "quantize_weight_int8", "op": "quantize", "M": 28672, "K": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(("experts", "experts", "experts", "linear", "linear", "quantize"))
    if op == "quantize":
        while True:
            M, K = _log_int(rng, 1, 28672), _log_int(rng, 64, 16384, 8)
            if M * K <= 28672 * 4096:
                break
        return {"op": op, "M": M, "K": K, "dtype": rng.choice(("bf16", "bf16", "f32"))}
    if op == "linear":
        while True:
            M, K = _log_int(rng, 1, 8192), _log_int(rng, 256, 8192, 16)
            n = [_log_int(rng, 256, 14336, 8) for _ in range(rng.randint(1, 3))] + [0, 0]
            if M * K * sum(n) <= 8192 * 4096 * 4096 and K * sum(n) <= 4096 * 28672:
                break
        return {"op": op, "M": M, "K": K, "n0": n[0], "n1": n[1], "n2": n[2], "L": rng.randint(1, 48),
                "runs": 0 if M <= 64 else rng.randint(1, 40)}
    while True:
        M, E = _log_int(rng, 1, 8192), _log_int(rng, 2, 128)
        K, N = _log_int(rng, 128, 14336, 16), _log_int(rng, 128, 28672, 8)
        topk = rng.randint(1, min(8, E))
        if M * topk * K * N <= 4096 * 2 * 14336 * 4096 and E * K * N <= 8 * 4096 * 28672:
            break
    return {"op": op, "M": M, "E": E, "topk": topk, "K": K, "N": N, "dtype": rng.choice(("bf16", "e4m3", "int8")),
            "pair_rows": rng.random() < 0.5, "skew": rng.choice((0.0, 0.3, 1.0, 2.0))}


def _touched(n, p, M):
    """Expected number of n equally likely choices taken by M tokens, each with probability p."""
    return n * (1.0 - (1.0 - p) ** M)


def _ranks(case):
    return [RANKS[i % len(RANKS)] for i in range(case["L"])]


def _slices(case):
    return [n for n in (case["n0"], case["n1"], case["n2"]) if n]


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantize":
        s = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * K * (s + 1) + 4 * M, "flops": 3 * M * K}
    if case["op"] == "linear":
        N, n_sl, L = sum(_slices(case)), len(_slices(case)), case["L"]
        rank = sum(_ranks(case)) / L
        tokens = M * (L / (L + 1.0)) * (1 - _ranks(case).count(0) / L)
        groups = M if case["runs"] == 0 else min(M, case["runs"])
        used = _touched(L, 1.0 / (L + 1), groups)
        return {"bytes": N * K + 4 * N + M * K + 4 * M + 2 * tokens * K + 2 * M * N + used * rank * 2 * (n_sl * K + N),
                "flops": 2 * M * N * K + 2 * tokens * rank * (n_sl * K + N)}
    E, topk, N = case["E"], case["topk"], case["N"]
    P = M * topk
    width = 2 if case["dtype"] == "bf16" else 1
    rows = P if case["pair_rows"] else M
    scales = 0 if width == 2 else 4 * rows + 4 * N * _touched(E, topk / E, M)
    return {"bytes": _touched(E, topk / E, M) * N * K * width + rows * K * width + 2 * P * N + 8 * P + 4 * (E + 1) + scales,
            "flops": 2 * P * N * K}


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _eight_bits(t, kind):
    """Rows in 8 bits with one scale each, as a checkpoint holds them."""
    top = 448.0 if kind == "e4m3" else INT8_MAX
    s = t.float().abs().amax(-1).clamp_min(1e-12) / top
    v = (t.float() / s[..., None]).clamp(-top, top)
    return (v.to(E4M3) if kind == "e4m3" else v.round().to(torch.int8)), s


def _make(case, seed):
    """The inputs as plain tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * std).to(dtype)

    M, K = case["M"], case["K"]
    if case["op"] == "quantize":
        s = {"x": randn(M, K, dtype=_dtype(case))}
        s["x"][:, ::61] *= 20.0         # the few large channels of real activations
        return s
    if case["op"] == "linear":
        L, sizes = case["L"], _slices(case)
        N, n_sl, ranks = sum(sizes), len(sizes), _ranks(case)
        s = {"x": randn(M, K)}
        s["x8"], s["xs"] = _eight_bits(s["x"], "int8")
        s["W8"], s["ws"] = _eight_bits(randn(N, K, std=0.02), "int8")
        s["A"] = [randn(n_sl * r, K, std=0.02) for r in ranks]
        s["B"] = [randn(N, r, std=0.02) for r in ranks]
        if case["runs"]:                # one id for each sequence of the batch
            pick = torch.randint(-1, L, (case["runs"],), generator=g, device="cuda")
            cuts = torch.randint(0, M, (case["runs"] - 1,), generator=g, device="cuda").sort().values
            s["ids"] = pick[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)].int()
        else:
            s["ids"] = torch.randint(-1, L, (M,), generator=g, device="cuda").int()
        return s
    E, N, topk = case["E"], case["N"], case["topk"]
    # a router's choice: different experts for each token, some liked more than others
    logits = randn(M, E, dtype=torch.float32) + case["skew"] * randn(E, dtype=torch.float32)
    s = {"topk_ids": torch.topk(logits, topk, dim=1).indices.int(), "xs": None, "ws": None}
    if case["pair_rows"]:               # what the activation leaves
        gate, up = randn(M * topk, K), randn(M * topk, K)
        s["x"] = gate * torch.sigmoid(gate) * up
    else:
        s["x"] = randn(M, K)
    if case["dtype"] == "bf16":
        s["W"] = randn(E, N, K, std=0.02)
        return s
    s["x"], s["xs"] = _eight_bits(s["x"], case["dtype"])
    s["W"] = torch.empty(E, N, K, dtype=s["x"].dtype, device="cuda")
    s["ws"] = torch.empty(E, N, dtype=torch.float32, device="cuda")
    for e in range(E):
        s["W"][e], s["ws"][e] = _eight_bits(randn(N, K, std=0.02), case["dtype"])
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    M, K = case["M"], case["K"]
    if case["op"] == "linear":          # every adapter padded to one rank, for the plain form
        ranks, sizes = _ranks(case), _slices(case)
        r, n_sl, N = 64, len(sizes), sum(sizes)
        s["A_all"] = torch.zeros(case["L"], n_sl, r, K, dtype=torch.bfloat16, device="cuda")
        s["B_all"] = torch.zeros(case["L"], N, r, dtype=torch.bfloat16, device="cuda")
        for i, q in enumerate(ranks):
            if q:
                s["A_all"][i, :, :q] = s["A"][i].view(n_sl, q, K)
                s["B_all"][i, :, :q] = s["B"][i]
        s["slice_of"] = torch.repeat_interleave(torch.arange(n_sl, device="cuda"), torch.tensor(sizes, device="cuda"))
    if own:
        import adapter_lora_amd as ml
        empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        if case["op"] == "quantize":
            s["out8"], s["scale"] = empty(M, K, dtype=torch.int8), empty(M, dtype=torch.float32)
        elif case["op"] == "linear":
            s["table"] = ml.LoraTable(s["A"], s["B"], _ranks(case), _slices(case), K, torch.bfloat16)
            s["seg"] = ml.Segments(M, case["L"])
            ml.lora_build_segments(s["ids"], s["seg"])
            s["wspace"] = ml.Workspace.for_table(s["table"], M)
            s["y"] = empty(M, s["table"].N, dtype=torch.bfloat16)
        else:
            s["groups"] = ml.MoeGroups(M * case["topk"], case["E"])
            s["y"] = empty(M * case["topk"], case["N"], dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass
def _run_own(s):
    import adapter_lora_amd as ml
    case = s["case"]
    if case["op"] == "quantize":
        ml.lora_quantize_rows(s["x"], s["out8"], s["scale"])
        return {"out8": s["out8"], "scale": s["scale"]}
    if case["op"] == "linear":
        ml.lora_linear_int8(s["table"], s["W8"], s["ws"], s["x8"], s["xs"], s["x"], s["seg"], s["y"], s["wspace"])
        return {"y": s["y"]}
    ml.lora_moe_group(s["topk_ids"], s["groups"])
    ml.lora_moe_linear(s["W"], s["x"], case["topk"], s["groups"], s["y"], w_scale=s["ws"], x_scale=s["xs"])
    return {"y": s["y"], "pairs": s["groups"].pairs, "offsets": s["groups"].offsets}


def _quantize_plain(x):
    # the scale is held in 32 bits; the quotient next to a border of two integers needs more
    top = x.float().abs().amax(1).double()
    scale = torch.where(top > 0, top / INT8_MAX, torch.ones_like(top)).float()
    return torch.round(x.double() / scale.double()[:, None]).to(torch.int8), scale


def _linear_plain(s):
    ids = s["ids"].long()
    L, n_sl, r, K = s["A_all"].shape
    base = (s["x8"].float() @ s["W8"].float().t()) * s["xs"][:, None] * s["ws"][None, :]
    S = (s["x"].float() @ s["A_all"].float().view(L * n_sl * r, K).t()).view(-1, L, n_sl, 1, r)
    mine = (ids[:, None] == torch.arange(L, device=ids.device)).view(-1, L, 1, 1, 1)
    # columns of other slices meet zeros: one product over (adapter, slice, rank)
    onto = (s["slice_of"][None, :] == torch.arange(n_sl, device=ids.device)[:, None]).float()      # [n_sl, N]
    B = s["B_all"].float().permute(0, 2, 1)[:, None] * onto[None, :, None]                         # [L, n_sl, r, N]
    return {"y": (base + (S * mine).reshape(-1, L * n_sl * r) @ B.reshape(L * n_sl * r, -1)).to(torch.bfloat16)}


def _experts_plain(s):
    case, flat = s["case"], s["topk_ids"].reshape(-1).long()
    E, topk, P = case["E"], case["topk"], flat.shape[0]
    pairs = torch.sort(flat, stable=True).indices
    counts = (flat[None, :] == torch.arange(E, device=flat.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    y = torch.empty(P, case["N"], dtype=torch.bfloat16, device=flat.device)
    cut = offsets.tolist()              # each expert's product has the size of its share
    for e in range(E):
        if cut[e] == cut[e + 1]:
            continue
        f = pairs[cut[e]:cut[e + 1]]
        rows = f if case["pair_rows"] else f // topk
        v = s["x"][rows].float() @ s["W"][e].float().t()
        if s["ws"] is not None:
            v = v * s["xs"][rows][:, None] * s["ws"][e][None, :]
        y[f] = v.to(torch.bfloat16)
    return {"y": y, "pairs": pairs.int(), "offsets": offsets.int()}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "quantize":
        out8, scale = _quantize_plain(state["x"])
        return {"out8": out8, "scale": scale}
    return _linear_plain(state) if op == "linear" else _experts_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _make(case, seed)
    if case["op"] == "quantize":
        return {"out8": None, "scale": torch.linalg.vector_norm(s["x"].double(), ord=float("inf"), dim=1) / INT8_MAX}
    if case["op"] == "linear":
        # the dequantised factors, then each adapter's own tokens and slices
        x = s["x"].double()
        y = (s["x8"].double() * s["xs"].double()[:, None]) @ (s["W8"].double() * s["ws"].double()[:, None]).t()
        for i, r in enumerate(_ranks(case)):
            rows = (s["ids"] == i).nonzero()[:, 0]
            n0 = 0
            for sl, n in enumerate(_slices(case)):
                if r and rows.numel():
                    A, B = s["A"][i][sl * r:(sl + 1) * r].double(), s["B"][i][n0:n0 + n].double()
                    y[rows, n0:n0 + n] += (x[rows] @ A.t()) @ B.t()
                n0 += n
        return {"y": y}
    topk = case["topk"]
    y = torch.zeros(case["M"] * topk, case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):          # every token that chose the expert, wherever it did
        m, j = (s["topk_ids"] == e).nonzero(as_tuple=True)
        if m.numel() == 0:
            continue
        f = m * topk + j
        x, W = s["x"][f if case["pair_rows"] else m].double(), s["W"][e].double()
        if s["ws"] is not None:
            x, W = x * s["xs"][f if case["pair_rows"] else m].double()[:, None], W * s["ws"][e].double()[:, None]
        y[f] = x @ W.t()
    return {"y": y, "pairs": None, "offsets": None}
