"""lora_moe_decode against the 64-bit oracle.

Tolerance of one output: half a bf16 step (2^-8) for the output and for h,
and UNIT of the terms' magnitudes for each fp32 sum ((2 K + 256) 2^-24 for K
products in two serial sums, 2^-16 for S as a bf16 pair), carried through the
layer by the oracle.  The routing the oracle is given is the kernel's own,
which is compared with the oracle's wherever two logits are not within the
rounding of their sums."""
import numpy as np
import pytest
import torch

from oracle import decoder as O

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F64 = lambda t: t.detach().double().cpu().numpy()     # noqa: E731


class Layer:
    def __init__(self, M, E, topk, H, I, L=2, r=16, w8=False, renorm=False, shared=False, ids=None,
                 seed=0, enabled=None):
        import adapter_lora_amd as ml
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, std=1.0):
            return (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()

        self.M, self.E, self.topk, self.H, self.I, self.L, self.renorm = M, E, topk, H, I, L, renorm
        self.x, self.router = rnd(M, H), rnd(E, H, std=H ** -0.5)
        self.W_gu, self.W_d = rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5)
        self.s_gu = self.s_d = None
        if w8:
            self.s_gu = torch.rand(E, 2 * I, generator=g, device="cuda") * 0.01 + 0.005
            self.s_d = torch.rand(E, H, generator=g, device="cuda") * 0.01 + 0.005
            self.W_gu = (self.W_gu.float() / self.s_gu[..., None]).clamp(-448, 448).to(E4M3)
            self.W_d = (self.W_d.float() / self.s_d[..., None]).clamp(-448, 448).to(E4M3)
        eo = 1 if shared else E
        self.adapters = None
        self.w = None
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda") if ids is not None else \
            torch.randint(-1, max(L, 1), (M,), generator=g, device="cuda").int()
        self.enabled = torch.ones(max(L, 1), dtype=torch.int32, device="cuda") if enabled is None \
            else torch.tensor(enabled, dtype=torch.int32, device="cuda")
        if L:
            self.adapters = (rnd(L, eo, r, H, std=0.05), rnd(L, E, 2 * I, r, std=0.3),
                             rnd(L, E, r, I, std=0.05), rnd(L, eo, H, r, std=0.3))
            self.w = ml.MoeWeights(*self.adapters, self.enabled)
        self.experts = ml.MoeExperts(self.router, self.W_gu, self.W_d, topk, renormalize=renorm,
                                     s_gu=self.s_gu, s_d=self.s_d)
        self.ws = ml.Workspace(ml.lora_moe_decode_workspace_size(self.w, self.experts, M))
        self.topk_ids = torch.full((M, topk), -7, dtype=torch.int32, device="cuda")
        self.topk_w = torch.empty(M, topk, device="cuda")

    def run(self, out=None, x=None, stream=None):
        import adapter_lora_amd as ml
        out = torch.full((self.M, self.H), float("nan"), dtype=torch.bfloat16, device="cuda") \
            if out is None else out
        ml.lora_moe_decode(self.w, self.experts, self.ids if self.w is not None else None,
                           self.x if x is None else x, out, self.ws, topk_ids=self.topk_ids,
                           topk_weights=self.topk_w, stream=stream)
        return out

    def check(self, out):
        import adapter_lora_amd as ml
        x, router = F64(self.x), F64(self.router)
        ids, w = self.topk_ids.cpu().numpy(), F64(self.topk_w)
        logits, mag = x @ router.T, np.abs(x) @ np.abs(router).T
        close = (self.H + 64) * 2.0 ** -24 * mag.max(1)
        want_ids, _ = O.route(x, router, self.topk, self.renorm)
        for m in range(self.M):
            assert len(set(ids[m])) == self.topk and (ids[m] >= 0).all() and (ids[m] < self.E).all()
            for k in range(self.topk):
                a, b = logits[m, ids[m, k]], logits[m, want_ids[m, k]]
                assert ids[m, k] == want_ids[m, k] or abs(a - b) <= 2 * close[m], (m, k)
        e = np.exp(logits - logits.max(1, keepdims=True))
        p = np.take_along_axis(e / e.sum(1, keepdims=True), ids, 1)
        if self.renorm:
            p = p / p.sum(1, keepdims=True)
        # exp of a logit off by `close`, a sum of E terms, a quotient
        assert (np.abs(w - p) <= p * (4 * close[:, None] + (self.E + 32) * 2.0 ** -24)).all()
        W_gu, W_d = F64(self.W_gu.float()), F64(self.W_d.float())
        if self.s_gu is not None:
            W_gu, W_d = W_gu * F64(self.s_gu)[..., None], W_d * F64(self.s_d)[..., None]
        unit = (2 * max(self.H, self.I) + 256) * 2.0 ** -24 + 2.0 ** -16
        ad = None if self.adapters is None else [F64(t) for t in self.adapters]
        want, bound = O.moe_layer_mag(x, ids, w, W_gu, W_d, self.ids.cpu().numpy(), ad,
                                      self.enabled.cpu().numpy(), 2.0 ** -8, unit)
        got = F64(out)
        bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1.02 * bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
        # and as a whole: two bf16 roundings make about 0.0024
        assert np.linalg.norm(got - want) <= 0.004 * np.linalg.norm(want)
        assert ml.lora_read_device_error(self.ws.buf) == 0


CASES = {
    "one_token": dict(M=1, E=8, topk=2, H=512, I=256),
    "one_expert": dict(M=3, E=1, topk=1, H=128, I=64),
    "smallest": dict(M=1, E=2, topk=1, H=8, I=8),
    "smallest_fp8": dict(M=2, E=2, topk=2, H=16, I=16, w8=True),
    "ragged": dict(M=17, E=5, topk=3, H=520, I=136, L=3, r=32),
    "ragged_fp8": dict(M=19, E=6, topk=2, H=528, I=144, L=3, r=64, w8=True, renorm=True),
    "no_adapters": dict(M=9, E=4, topk=2, H=256, I=192, L=0),
    "all_none": dict(M=6, E=4, topk=2, H=256, I=128, ids=[-1] * 6),
    "disabled_and_outside": dict(M=10, E=4, topk=2, H=256, I=128, L=3, enabled=[1, 0, 1],
                                 ids=[0, 1, 2, -1, 3, 99, -9, 0, 1, 2]),
    "shared_outer": dict(M=12, E=4, topk=2, H=320, I=192, L=3, r=32, shared=True),
    "every_expert": dict(M=40, E=16, topk=16, H=128, I=64, L=4),
    "one_busy_expert": dict(M=64, E=2, topk=1, H=256, I=128, L=1, ids=[0] * 64),
    "full_batch": dict(M=64, E=8, topk=2, H=384, I=320, L=5, r=16, renorm=True),
    "full_batch_fp8": dict(M=64, E=12, topk=4, H=256, I=208, L=8, r=32, w8=True),
    "many_experts": dict(M=33, E=256, topk=8, H=64, I=32, L=2),
    "long_inner": dict(M=4, E=3, topk=2, H=64, I=4104, L=2),
    "split_down": dict(M=30, E=4, topk=2, H=48, I=2048, L=3, r=64),
    "wide_hidden": dict(M=2, E=2, topk=1, H=4096, I=40, L=2),
}


@pytest.mark.parametrize("name", list(CASES))
def test_moe_decode_matches_oracle(name):
    print(name, flush=True)
    layer = Layer(**CASES[name])
    layer.check(layer.run())


def test_ties_go_to_the_lowest_expert():
    layer = Layer(M=5, E=12, topk=4, H=64, I=32)
    layer.router[3:].copy_(layer.router[3:4].expand(9, 64))      # nine equal rows
    layer.router[:3].zero_()                                     # and three equal zeros
    layer.run()
    logits = F64(layer.x) @ F64(layer.router).T
    for m in range(5):
        want = [3, 4, 5, 6] if logits[m, 3] > 0 else [0, 1, 2, 3]
        assert layer.topk_ids[m].tolist() == want


def test_strided_rows_and_neighbours():
    layer = Layer(M=21, E=4, topk=2, H=136, I=72, L=2)
    xw = torch.full((22, 136 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:21, 8:144] = layer.x
    ow = torch.full((22, 136 + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    layer.check(layer.run(out=ow[:21, 8:144], x=xw[:21, 8:144]))
    assert (ow[21] == 3).all() and (ow[:, :8] == 3).all() and (ow[:, 144:] == 3).all()


@pytest.mark.parametrize("w8", [False, True])
def test_repeats_bit_identical_on_one_workspace(w8):
    layer = Layer(M=37, E=6, topk=3, H=256, I=528, L=3, r=32, w8=w8)
    first = layer.run()
    side = torch.cuda.Stream()
    for i in range(6):
        torch.cuda.synchronize()
        again = layer.run(stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


def test_nan_stays_with_its_token():
    layer = Layer(M=18, E=4, topk=2, H=128, I=64)
    clean = layer.run()
    layer.x[7, 11] = float("nan")
    out = layer.run()
    assert torch.isnan(out[7]).all()
    rest = [m for m in range(18) if m != 7]
    assert torch.equal(out[rest], clean[rest])


def test_no_tokens():
    import adapter_lora_amd as ml
    layer = Layer(M=1, E=2, topk=1, H=64, I=32)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ml.lora_moe_decode(layer.w, layer.experts, layer.ids[:0], e, torch.empty_like(e), layer.ws)


def test_graph_replays_with_new_inputs():
    layer, other = Layer(M=13, E=8, topk=2, H=256, I=128, L=3), Layer(M=13, E=8, topk=2, H=256, I=128, seed=9)
    out = layer.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.run(out, stream=torch.cuda.current_stream())
    mine = layer.x.clone()
    for i in range(5):
        layer.x.copy_(other.x if i % 2 else mine)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer.run())
        torch.cuda.synchronize()
        layer.check(got)
