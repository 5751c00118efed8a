"""The decoder layer's 8-bit and MoE calls as they are used: norm, projection
beside the adapters, norm, MoE layer, in one queue of launches and in one
captured graph; workspaces that graphs share; infinities of one adapter or
expert; and the checked library."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import decoder as O
from tests.test_gpu_linear_fp8 import Case
from tests.test_gpu_moe_decode import Layer
from tests.test_gpu_rms_norm import HALF, UNIT, check_eight, near

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F64 = lambda t: t.detach().double().cpu().numpy()     # noqa: E731
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Chain:
    """attention output and residual -> norm -> projection -> norm -> MoE"""

    def __init__(self, M, H=528, seed=0, moe=True):
        import adapter_lora_amd as ml
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()     # noqa: E731
        self.M, self.H = M, H
        self.c = Case(M, H, [H - 16, 16], [16, 0, 64], None, seed=seed)
        W = rnd(H, H)
        ml.lora_quantize_rows(W, self.c.W8, self.c.ws)
        self.a, self.res = rnd(M, H), rnd(M, H)
        self.n1, self.n2 = rnd(H), rnd(H)
        self.res1, self.res2 = torch.empty_like(self.res), torch.empty_like(self.res)
        self.y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
        self.moe = Layer(M=M, E=6, topk=2, H=H, I=144, L=3, r=32, w8=True, ids=self.c.ids.tolist(),
                         seed=seed) if moe else None
        self.normed = self.moe.x if moe else torch.empty_like(self.y)
        self.out = torch.empty_like(self.y)

    def run(self):
        import adapter_lora_amd as ml
        c = self.c
        ml.lora_build_segments(c.ids, c.seg)
        ml.lora_rms_norm(self.a, self.n1, 1e-5, residual=self.res, residual_out=self.res1, out=c.x,
                         out8=c.x8, scale=c.xs)
        c.run(self.y)
        ml.lora_rms_norm(self.y, self.n2, 1e-5, residual=self.res1, residual_out=self.res2,
                         out=self.normed)
        if self.moe:
            self.moe.run(self.out)
        return [t.clone() for t in (self.y, self.res2, self.normed)] + \
            ([self.out.clone()] if self.moe else [])

    def check(self):
        """Each call against the 64-bit oracle on what it was given."""
        h, v = O.rms_norm(F64(self.a), F64(self.n1), 1e-5, F64(self.res))
        near(F64(self.res1), h, HALF[torch.bfloat16] * 1.0001, what="residual 1")
        near(F64(self.c.x), v, HALF[torch.bfloat16] + UNIT, what="norm 1")
        check_eight(self.c.x8, self.c.xs, v, "norm 1")
        self.c.check(self.y)
        h, v = O.rms_norm(F64(self.y), F64(self.n2), 1e-5, F64(self.res1))
        near(F64(self.res2), h, HALF[torch.bfloat16] * 1.0001, what="residual 2")
        near(F64(self.normed), v, HALF[torch.bfloat16] + UNIT, what="norm 2")
        if self.moe:
            self.moe.check(self.out)


@pytest.mark.parametrize("M,moe", [(1, True), (37, True), (64, True), (65, False), (300, False)])
def test_layer_in_one_queue(M, moe):
    print(M, flush=True)
    c = Chain(M, seed=M, moe=moe)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_layer_captured_and_replayed():
    c, d = Chain(21, seed=1), Chain(21, seed=2)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    mine = c.a.clone(), c.res.clone(), c.c.ids.clone()
    for i in range(5):
        src = (d.a, d.res, d.c.ids) if i % 2 else mine
        for to, t in zip((c.a, c.res, c.c.ids), src):
            to.copy_(t)
        c.moe.ids.copy_(c.c.ids)
        c.out.zero_(), c.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.y, c.res2, c.normed, c.out)]
        c.check()
        eager = c.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_two_graphs_share_a_workspace():
    """Two captured graphs of different sizes whose calls use one workspace,
    replayed in turn on one stream: each replay equals its eager result."""
    import adapter_lora_amd as ml
    big, small = Case(64, 1040, [264], [16, 64], None, seed=1), Case(9, 1040, [264], [64, 16], None, seed=2)
    lb = Layer(M=64, E=5, topk=2, H=256, I=144, L=3, r=32, seed=3)
    ls = Layer(M=5, E=5, topk=2, H=256, I=144, L=3, r=32, seed=4)
    assert ls.ws.nbytes <= lb.ws.nbytes
    small.ws_buf, ls.ws = big.ws_buf, lb.ws
    users = [big, small, lb, ls]
    want, graphs, outs = [], [], []
    for u in users:
        want.append(u.run())
        u.check(want[-1])
        torch.cuda.synchronize()
        outs.append(torch.zeros_like(want[-1]))
    for u, o in zip(users, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            u.run(o)
        graphs.append(g)
    for i in (0, 1, 1, 0, 2, 3, 3, 2, 0, 3):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i]), i
        assert torch.equal(users[i].run(), want[i])
        torch.cuda.synchronize()
    assert ml.lora_read_device_error(big.ws_buf.buf) == 0 and ml.lora_read_device_error(lb.ws.buf) == 0


@pytest.mark.parametrize("M,K,sizes", [(40, 512, [72]), (64, 4096, [16]), (200, 2064, [264, 40]),
                                       (300, 1040, [264, 72]), (300, 144, [13320])])
def test_adapters_infinities_stay_with_its_tokens(M, K, sizes):
    """Infinite and NaN values in one adapter's B make its own tokens' columns
    infinite or NaN, a NaN in its A all its outputs; everything else keeps its
    bits."""
    import adapter_lora_amd as ml
    c = Case(M, K, sizes, [16, 32, 64], None, seed=5)
    clean = c.run()
    c.check(clean)
    c.B[1][3, 1] = float("inf")
    c.B[1][5, 0] = float("nan")
    c.B[1][6, 31] = float("-inf")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    y = c.run()
    other = c.ids != 1
    assert other.any() and (~other).any()
    assert torch.equal(y[other], clean[other])
    # S enters as hi + lo: inf * hi + inf * lo is NaN where their signs differ,
    # so an infinite column is promised to be infinite or NaN, no more
    assert not torch.isfinite(y[~other][:, [3, 5, 6]]).any()
    rest = [n for n in range(c.N) if n not in (3, 5, 6)]
    assert torch.equal(y[~other][:, rest], clean[~other][:, rest])
    c.A[1][2, 7] = float("nan")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    y = c.run()
    assert torch.equal(y[other], clean[other])
    assert torch.isnan(y[~other][:, :sizes[0]]).all()


@pytest.mark.parametrize("M,w8", [(6, False), (14, True), (30, False), (30, True), (60, False)])
def test_experts_infinities_stay_with_its_tokens(M, w8):
    """The same of one expert (in 8 bits NaN alone, e4m3 has no infinities)."""
    layer = Layer(M=M, E=6, topk=2, H=144, I=80, L=3, r=16, w8=w8, seed=M)
    clean = layer.run()
    layer.check(clean)
    e = int(layer.topk_ids[0, 0])
    other = (layer.topk_ids != e).all(1)
    assert other.any()
    if w8:
        layer.W_d.view(torch.uint8)[e, 9, 4] = 0x7f
        layer.W_gu.view(torch.uint8)[e, 11, 3] = 0x7f
    else:
        layer.W_d[e, 9, 4] = float("inf")
        layer.W_gu[e, 11, 3] = float("nan")
    out = layer.run()
    assert torch.equal(out[other], clean[other])
    assert torch.isnan(out[~other]).any(1).all()


@pytest.mark.parametrize("which", [1, 3])
def test_moe_adapters_infinities_stay_with_its_tokens(which):
    layer = Layer(M=45, E=4, topk=2, H=144, I=80, L=3, r=32, ids=[0, 1, 2, -1, 1] * 9, seed=11)
    clean = layer.run()
    layer.check(clean)
    t = layer.adapters[which]                  # B_gu or B_d
    t[1, :, 3, 5] = float("inf")
    t[1, :, 6, 2] = float("nan")
    out = layer.run()
    other = layer.ids != 1
    assert torch.equal(out[other], clean[other])
    assert torch.isnan(out[~other]).any(1).all()


def child(fault):
    lib = os.path.join(ROOT, "adapter_lora_amd", "libmlora_debug.so")
    assert os.path.exists(lib), "run __graft_entry__.build() first"
    env = dict(os.environ, MLORA_LIB=lib)
    if fault:
        env["MLORA_DEBUG_WAIT_FAULT"] = "1"
    print("checked library, forced misses:", fault, flush=True)
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "debug_decoder_run.py")],
                       env=env, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["lib"] == "libmlora_debug.so"
    return res


def test_checked_library_tables():
    res = child(False)
    for name in ("decode", "groups", "product"):
        v = res[name]
        assert v["valid_err"] == 0 and v["valid_exact"], (name, v)
        assert v["err"] == 4 and v["padding_untouched"] and v["others_exact"], (name, v)  # LORA_DEVERR_TABLE
    assert res["moe_err"] == 0 and res["moe_same"], res


def test_checked_library_lost_waits_are_reported():
    res = child(True)
    assert res["decode"]["valid_err"] & 1 and res["moe_err"] & 1, res        # LORA_DEVERR_WAIT


@pytest.mark.parametrize("kw", [
    dict(M=64, E=256, topk=16, H=64, I=32, L=8, r=64),                  # every limit; S past the LDS copy
    dict(M=64, E=256, topk=16, H=32, I=48, L=3, r=16, w8=True, renorm=True),
    dict(M=64, E=3, topk=3, H=80, I=48, L=4, r=48, w8=True),            # two groups of every expert
    dict(M=33, E=2, topk=1, H=136, I=8, L=1, r=32),
    dict(M=8, E=64, topk=2, H=8, I=1000, L=2, r=64),
])
def test_moe_limits(kw):
    print(kw, flush=True)
    layer = Layer(**kw)
    layer.check(layer.run())


def test_experts_past_four_gigabytes():
    """20 experts of 235 MB each: every token goes to the last one, whose
    output has the bits of a layer that holds it alone (renormalized, so the
    routing weight is 1 in both)."""
    import adapter_lora_amd as ml
    E, H, I = 20, 4096, 9560
    small = Layer(M=5, E=1, topk=1, H=H, I=I, L=0, renorm=True)
    W_gu = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    W_d = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    W_gu[E - 1], W_d[E - 1] = small.W_gu[0], small.W_d[0]
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    router[:E - 1, 0] = -1000.0
    x = small.x
    x[:, 0] = 1.0
    want = small.run()
    ex = ml.MoeExperts(router, W_gu, W_d, 1, renormalize=True)
    ws = ml.Workspace(ml.lora_moe_decode_workspace_size(None, ex, 5))
    out = torch.empty_like(want)
    ids = torch.empty(5, 1, dtype=torch.int32, device="cuda")
    ml.lora_moe_decode(None, ex, None, x, out, ws, topk_ids=ids)
    torch.cuda.synchronize()
    assert W_gu.numel() * 2 > 1 << 31 and (W_gu.numel() + W_d.numel()) * 2 > 1 << 32
    assert (ids == E - 1).all() and torch.equal(out, want)


@pytest.mark.parametrize("M", [20, 100])
def test_rows_far_apart(M):
    """Rows of W8, x8 and x millions of values apart: offsets past 32 bits."""
    c = Case(M, 256, [264, 256], [16, 32], None, seed=9)
    want = c.run()
    c.check(want)

    def far(t, ld):
        buf = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=torch.uint8 if t.dtype == E4M3
                          else t.dtype, device="cuda")
        v = buf.view(t.dtype).as_strided(t.shape, (ld, 1))
        (v.view(torch.uint8) if t.dtype == E4M3 else v).copy_(t.view(torch.uint8) if t.dtype == E4M3 else t)
        return v

    W8 = far(c.W8, 8388576)                                   # 520 rows: 4.3 GB
    assert 519 * 8388576 > 1 << 32
    wide = 50_000_000 if M > 64 else 1 << 20                  # 99 rows: 4.95 GB
    x8 = far(c.x8, wide)
    x = far(c.x, wide // 2)
    assert torch.equal(c.run(x8=x8, W8=W8, x=x), want)


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams, many in flight."""
    a, b = Case(48, 2064, [264], [16, 64], None, seed=1), Layer(M=20, E=6, topk=2, H=528, I=400, L=3, r=32, w8=True)
    wa, wb = a.run(), b.run()
    a.check(wa), b.check(wb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ya, yb = [torch.zeros_like(wa) for _ in range(20)], [torch.zeros_like(wb) for _ in range(20)]
    torch.cuda.synchronize()
    for y, z in zip(ya, yb):
        a.run(y, stream=sa)
        b.run(z, stream=sb)
    torch.cuda.synchronize()
    assert all(torch.equal(y, wa) for y in ya) and all(torch.equal(z, wb) for z in yb)
