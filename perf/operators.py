"""The operators of one decoder layer in 8 bits beside its adapters: what is measured.

Three operators, in the order a layer runs them:

  * ``norm``: the residual's addition, the root-mean-square norm and its output
    in 8 bits with one scale per row (and the same kernel without the norm, for
    weights at load time and for activations that no norm precedes);
  * ``linear``: a shared projection held in 8 bits beside the adapters of many
    requests, y = (x8 W8^T) xs ws + (x A_i^T) B_i^T, from one token to prefill;
  * ``moe``: a whole mixture-of-experts layer for a few tokens, router, experts
    and their adapters, with experts in bf16 or in 8 bits with a scale per row.

Sizes: the repository's decode, prefill, stacked and MoE workloads (hidden size
4096, outputs 4096, [4096, 1024, 1024] and [14336, 14336], 8 experts of 14336,
top-2) and generic ones.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
RANKS = (16, 32, 64, 8, 20, 0)      # adapter ranks, in turn (0: an empty slot)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the norm before a projection while 32 requests decode: latency counts
        {"name": "norm_decode_32", "op": "norm", "M": 32, "K": 4096, "dtype": "bf16", "residual": True, "out": True, "out8": True},
        # the same norm over a prefill batch
        {"name": "norm_prefill_2048", "op": "norm", "M": 2048, "K": 4096, "dtype": "bf16", "residual": True, "out": True, "out8": True},
        # a final norm in fp32 over a ragged batch and an odd width, no 8-bit output
        {"name": "norm_ragged_fp32", "op": "norm", "M": 4099, "K": 5128, "dtype": "f32", "residual": False, "out": True, "out8": False},
        # the activations before the down projection of 64 tokens: 8 bits, no norm
        {"name": "quantize_act_64", "op": "quantize", "M": 64, "K": 14336, "dtype": "bf16"},
        # a gate/up weight brought to 8 bits at load time
        {"name": "quantize_weight", "op": "quantize", "M": 28672, "K": 4096, "dtype": "bf16"},
        # one token through the stacked query/key/value projection
        {"name": "linear_1_qkv", "op": "linear", "M": 1, "K": 4096, "n0": 4096, "n1": 1024, "n2": 1024, "L": 32, "runs": 0},
        # 32 decoding requests, each with an adapter of its own choice
        {"name": "linear_32", "op": "linear", "M": 32, "K": 4096, "n0": 4096, "n1": 0, "n2": 0, "L": 32, "runs": 0},
        # a mixed batch of 512 tokens through the stacked gate/up projection
        {"name": "linear_512_gate_up", "op": "linear", "M": 512, "K": 4096, "n0": 14336, "n1": 14336, "n2": 0, "L": 12, "runs": 36},
        # a prefill batch, one adapter per sequence
        {"name": "linear_2048", "op": "linear", "M": 2048, "K": 4096, "n0": 4096, "n1": 0, "n2": 0, "L": 8, "runs": 8},
        # one token through 2 of 8 large experts
        {"name": "moe_1", "op": "moe", "M": 1, "E": 8, "topk": 2, "H": 4096, "I": 14336, "L": 4, "r": 16, "w8": False, "renorm": False},
        # 27 tokens over many small experts in 8 bits, ragged widths
        {"name": "moe_27_fp8", "op": "moe", "M": 27, "E": 40, "topk": 4, "H": 2064, "I": 1424, "L": 6, "r": 32, "w8": True, "renorm": True},
        # the most tokens of one call: every expert is read
        {"name": "moe_64", "op": "moe", "M": 64, "E": 8, "topk": 2, "H": 4096, "I": 14336, "L": 4, "r": 16, "w8": False, "renorm": False},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(("norm", "quantize", "linear", "linear", "moe", "moe"))
    if op in ("norm", "quantize"):
        while True:
            M, K = _log_int(rng, 1, 28672), _log_int(rng, 64, 16384, 8)
            if M * K <= 28672 * 4096:
                break
        case = {"op": op, "M": M, "K": K, "dtype": rng.choice(("bf16", "bf16", "f32"))}
        if op == "norm":
            out8 = rng.random() < 0.7
            case.update(residual=rng.random() < 0.6, out=not out8 or rng.random() < 0.6, out8=out8)
        return case
    if op == "linear":
        while True:
            M, K = _log_int(rng, 1, 2048), _log_int(rng, 256, 8192, 16)
            n = [_log_int(rng, 256, 14336, 8) for _ in range(rng.randint(1, 3))] + [0, 0]
            if M * K * sum(n) <= 512 * 4096 * 28672 and K * sum(n) <= 4096 * 28672:
                break
        return {"op": op, "M": M, "K": K, "n0": n[0], "n1": n[1], "n2": n[2], "L": rng.randint(1, 48),
                "runs": 0 if M <= 64 else rng.randint(1, 40)}
    while True:
        M, E = _log_int(rng, 1, 64), _log_int(rng, 2, 64)
        H, I = _log_int(rng, 256, 4096, 16), _log_int(rng, 128, 14336, 16)
        if E * H * I <= 5 * 4096 * 14336:      # the adapters come on top
            break
    return {"op": op, "M": M, "E": E, "topk": rng.randint(1, min(8, E)), "H": H, "I": I, "L": rng.randint(1, 8),
            "r": rng.choice((16, 32, 64)), "w8": rng.random() < 0.5, "renorm": rng.random() < 0.5}


def _touched(n, p, M):
    """Expected number of n equally likely choices taken by M tokens, each with probability p."""
    return n * (1.0 - (1.0 - p) ** M)


def _ranks(case):
    return [RANKS[i % len(RANKS)] for i in range(case["L"])]


def _slices(case):
    return [n for n in (case["n0"], case["n1"], case["n2"]) if n]


def work(case):
    M = case["M"]
    if case["op"] in ("norm", "quantize"):
        K, s = case["K"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "quantize":
            return {"bytes": M * K * (s + 1) + 4 * M, "flops": 3 * M * K}
        per = s * (1 + 2 * case["residual"] + case["out"]) + case["out8"]
        return {"bytes": M * K * per + K * s + 4 * M * case["out8"], "flops": 6 * M * K}
    if case["op"] == "linear":
        K, N, n_sl, L = case["K"], sum(_slices(case)), len(_slices(case)), case["L"]
        rank = sum(_ranks(case)) / L
        tokens = M * (L / (L + 1.0)) * (1 - _ranks(case).count(0) / L)
        groups = M if case["runs"] == 0 else min(M, case["runs"])
        used = _touched(L, 1.0 / (L + 1), groups)
        return {"bytes": N * K + 4 * N + M * K + 4 * M + 2 * tokens * K + 2 * M * N + used * rank * 2 * (n_sl * K + N),
                "flops": 2 * M * N * K + 2 * tokens * rank * (n_sl * K + N)}
    E, k, H, I, L, r = (case[q] for q in ("E", "topk", "H", "I", "L", "r"))
    experts = _touched(E, k / E, M)
    pairs = M * k * L / (L + 1.0)
    slots = _touched(L * E, k / E / (L + 1.0), M)
    width = 1 if case["w8"] else 2
    adapters = slots * r * 2 * (H + 2 * I + I + H)
    return {"bytes": experts * 3 * H * I * width + (experts * 4 * (2 * I + H) if case["w8"] else 0) + 2 * E * H + 4 * M * H + adapters
            + 8 * M * k,
            "flops": 2 * M * E * H + 2 * M * k * 3 * H * I + 2 * pairs * r * (H + 2 * I + I + H)}


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _eight_bits(t):
    """Rows in 8 bits with one scale each, as a checkpoint holds them."""
    s = t.float().abs().amax(-1).clamp_min(1e-12) / E4M3_MAX
    return (t.float() / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _make(case, seed):
    """The inputs as plain tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * std).to(dtype)

    M, dt = case["M"], _dtype(case)
    if case["op"] in ("norm", "quantize"):
        K = case["K"]
        s = {"x": randn(M, K, dtype=dt)}
        s["x"][:, ::61] *= 20.0         # the few large channels of real activations
        if case["op"] == "norm":
            s["weight"] = (1.0 + 0.1 * randn(K, dtype=torch.float32)).to(dt)
            s["residual"] = randn(M, K, std=3.0, dtype=dt) if case["residual"] else None
        return s
    L = case["L"]
    if case["op"] == "linear":
        K, sizes = case["K"], _slices(case)
        N, n_sl, ranks = sum(sizes), len(sizes), _ranks(case)
        s = {"x": randn(M, K)}
        s["x8"], s["xs"] = _eight_bits(s["x"])
        s["W8"], s["ws"] = _eight_bits(randn(N, K, std=0.02))
        s["A"] = [randn(n_sl * r, K, std=0.02) for r in ranks]
        s["B"] = [randn(N, r, std=0.02) for r in ranks]
        if case["runs"]:                # one id for each sequence of the batch
            pick = torch.randint(-1, L, (case["runs"],), generator=g, device="cuda")
            cuts = torch.randint(0, M, (case["runs"] - 1,), generator=g, device="cuda").sort().values
            s["ids"] = pick[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)].int()
        else:
            s["ids"] = torch.randint(-1, L, (M,), generator=g, device="cuda").int()
        return s
    E, H, I, r = (case[q] for q in ("E", "H", "I", "r"))
    s = {"x": randn(M, H), "router": randn(E, H, std=0.02), "W_gu": randn(E, 2 * I, H, std=0.02), "W_d": randn(E, H, I, std=0.02),
         "s_gu": None, "s_d": None}
    if case["w8"]:
        s["W_gu"], s["s_gu"] = _eight_bits(s["W_gu"])
        s["W_d"], s["s_d"] = _eight_bits(s["W_d"])
    s.update(A_gu=randn(L, E, r, H, std=0.02), B_gu=randn(L, E, 2 * I, r, std=0.02), A_d=randn(L, E, r, I, std=0.02),
             B_d=randn(L, E, H, r, std=0.02), ids=torch.randint(-1, L, (M,), generator=g, device="cuda").int())
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    M, dt = case["M"], _dtype(case)
    if case["op"] == "linear":          # every adapter padded to one rank, for the plain form
        ranks, sizes = _ranks(case), _slices(case)
        r, n_sl, N, K = 64, len(sizes), sum(sizes), case["K"]
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
        if case["op"] in ("norm", "quantize"):
            K, q = case["K"], case["op"] == "quantize"
            eight = q or case["out8"]
            s["out"] = empty(M, K, dtype=dt) if not q and case["out"] else None
            s["out8"] = empty(M, K, dtype=E4M3) if eight else None
            s["scale"] = empty(M, dtype=torch.float32) if eight else None
            s["residual_out"] = empty(M, K, dtype=dt) if s.get("residual") is not None else None
        elif case["op"] == "linear":
            ranks = _ranks(case)
            s["table"] = ml.LoraTable(s["A"], s["B"], ranks, _slices(case), case["K"], torch.bfloat16)
            s["seg"] = ml.Segments(M, case["L"])
            ml.lora_build_segments(s["ids"], s["seg"])
            s["wspace"] = ml.Workspace.for_table(s["table"], M)
            s["y"] = empty(M, s["table"].N, dtype=torch.bfloat16)
        else:
            on = torch.ones(case["L"], dtype=torch.int32, device="cuda")
            s["adapters"] = ml.MoeWeights(s["A_gu"], s["B_gu"], s["A_d"], s["B_d"], on)
            s["experts"] = ml.MoeExperts(s["router"], s["W_gu"], s["W_d"], case["topk"], renormalize=case["renorm"],
                                         s_gu=s["s_gu"], s_d=s["s_d"])
            s["wspace"] = ml.Workspace(ml.lora_moe_decode_workspace_size(s["adapters"], s["experts"], M))
            s["out"] = empty(M, case["H"], dtype=torch.bfloat16)
            s["topk_ids"] = empty(M, case["topk"], dtype=torch.int32)
            s["topk_weights"] = empty(M, case["topk"], dtype=torch.float32)
    return s


# ---------------------------------------------------------------- one pass
EPS = 1e-6


def _run_own(s):
    import adapter_lora_amd as ml
    case = s["case"]
    if case["op"] == "norm":
        ml.lora_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], out=s["out"],
                         out8=s["out8"], scale=s["scale"])
        return {"out": s["out"], "out8": s["out8"], "scale": s["scale"], "residual": s["residual_out"]}
    if case["op"] == "quantize":
        ml.lora_quantize_rows(s["x"], s["out8"], s["scale"])
        return {"out8": s["out8"], "scale": s["scale"]}
    if case["op"] == "linear":
        ml.lora_linear_fp8(s["table"], s["W8"], s["ws"], s["x8"], s["xs"], s["x"], s["seg"], s["y"], s["wspace"])
        return {"y": s["y"]}
    ml.lora_moe_decode(s["adapters"], s["experts"], s["ids"], s["x"], s["out"], s["wspace"], topk_ids=s["topk_ids"],
                       topk_weights=s["topk_weights"])
    return {"out": s["out"], "topk_ids": s["topk_ids"], "topk_weights": s["topk_weights"]}


def _quantize_plain(v):
    top = v.abs().amax(1)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def _norm_plain(s):
    case, dt = s["case"], s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    out8, scale = _quantize_plain(v) if case["out8"] else (None, None)
    return {"out": v.to(dt) if case["out"] else None, "out8": out8, "scale": scale,
            "residual": h.to(dt) if s["residual"] is not None else None}


def _linear_plain(s):
    case, ids = s["case"], s["ids"].long()
    L, n_sl, r, K = s["A_all"].shape
    base = (s["x8"].float() @ s["W8"].float().t()) * s["xs"][:, None] * s["ws"][None, :]
    S = (s["x"].float() @ s["A_all"].float().view(L * n_sl * r, K).t()).view(-1, L, n_sl, 1, r)
    mine = (ids[:, None] == torch.arange(L, device=ids.device)).view(-1, L, 1, 1, 1)
    # columns of other slices meet zeros: one product over (adapter, slice, rank)
    onto = (s["slice_of"][None, :] == torch.arange(n_sl, device=ids.device)[:, None]).float()      # [n_sl, N]
    B = s["B_all"].float().permute(0, 2, 1)[:, None] * onto[None, :, None]                         # [L, n_sl, r, N]
    return {"y": (base + (S * mine).reshape(-1, L * n_sl * r) @ B.reshape(L * n_sl * r, -1)).to(torch.bfloat16)}


def _moe_plain(s):
    case, x, ids = s["case"], s["x"].float(), s["ids"].long()
    E, k, I, L, r = (case[q] for q in ("E", "topk", "I", "L", "r"))
    M = x.shape[0]
    p = torch.softmax(x @ s["router"].float().t(), 1)
    top, order = torch.sort(p, dim=1, descending=True, stable=True)
    weights, experts = top[:, :k], order[:, :k]
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    W_gu, W_d = s["W_gu"].float(), s["W_d"].float()
    if s["s_gu"] is not None:
        W_gu, W_d = W_gu * s["s_gu"][..., None], W_d * s["s_d"][..., None]
    rows = torch.arange(M, device=x.device)[:, None].expand(M, k)
    on = (ids >= 0)[:, None, None].float()
    pick = ids.clamp_min(0)[:, None].expand(M, k)
    A_gu, B_gu = s["A_gu"][pick, experts].float(), s["B_gu"][pick, experts].float()                # [M, k, r, H], [M, k, 2I, r]
    A_d, B_d = s["A_d"][pick, experts].float(), s["B_d"][pick, experts].float()
    S = (A_gu @ x[:, None, :, None])                                                              # [M, k, r, 1]
    gu = (x[None] @ W_gu.transpose(1, 2))[experts, rows] + (B_gu @ S)[..., 0] * on
    h = gu[..., :I] / (1 + torch.exp(-gu[..., :I])) * gu[..., I:]
    S = A_d @ h[..., None]
    # every pair's row stands in its expert's batch, zeros elsewhere
    spread = torch.zeros(E, M, I, device=x.device).index_put((experts, rows), h * weights[..., None])
    out = (spread @ W_d.transpose(1, 2)).sum(0) + (((B_d @ S)[..., 0] * on) * weights[..., None]).sum(1)
    return {"out": out.to(torch.bfloat16), "topk_ids": experts.int(), "topk_weights": weights}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "quantize":
        out8, scale = _quantize_plain(state["x"].float())
        return {"out8": out8, "scale": scale}
    return _linear_plain(state) if op == "linear" else _moe_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _make(case, seed)
    x = s["x"].double()
    if case["op"] in ("norm", "quantize"):
        res = s.get("residual")
        h = x if res is None else x + res.double()
        v = h
        if case["op"] == "norm":
            v = h / torch.sqrt(torch.linalg.vecdot(h, h)[:, None] / case["K"] + EPS) * s["weight"].double()
        eight = case["op"] == "quantize" or case["out8"]
        scale = torch.linalg.vector_norm(v, ord=float("inf"), dim=1) / E4M3_MAX
        got = {"out8": v / scale[:, None] if eight else None, "scale": scale if eight else None}
        if case["op"] == "norm":
            got.update(out=v if case["out"] else None, residual=None if res is None else h)
        return got
    if case["op"] == "linear":
        # the dequantised factors, then each adapter's own tokens and slices
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
    k, I, M = case["topk"], case["I"], case["M"]
    logits = x @ s["router"].double().t()
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    weights = torch.empty(M, k, dtype=torch.float64, device="cuda")
    left = p.clone()
    for j in range(k):                  # the largest of what is left, the lowest index of equals
        at = (left == left.max(1, keepdim=True).values).int().argmax(1)
        ids[:, j], weights[:, j] = at.int(), p.gather(1, at[:, None])[:, 0]
        left.scatter_(1, at[:, None], -1.0)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    out = torch.zeros(M, case["H"], dtype=torch.float64, device="cuda")
    for n in range(case["E"]):          # an expert at a time, its weights in 64 bits
        rows, place = (ids == n).nonzero(as_tuple=True)
        if rows.numel() == 0:
            continue
        W_gu, W_d = s["W_gu"][n].double(), s["W_d"][n].double()
        if case["w8"]:
            W_gu, W_d = W_gu * s["s_gu"][n].double()[:, None], W_d * s["s_d"][n].double()[:, None]
        for a in [-1] + list(range(case["L"])):
            sel = s["ids"][rows] == a
            if not bool(sel.any()):
                continue
            t, w = rows[sel], weights[rows[sel], place[sel]]
            G, D = W_gu, W_d
            if a >= 0:                  # the adapter merged into the expert
                G = G + s["B_gu"][a, n].double() @ s["A_gu"][a, n].double()
                D = D + s["B_d"][a, n].double() @ s["A_d"][a, n].double()
            gu = x[t] @ G.t()
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            out.index_add_(0, t, (h @ D.t()) * w[:, None])
    return {"out": out, "topk_ids": None, "topk_weights": weights}
