"""Refusals of the 8-bit decoder-layer calls (before any launch, no GPU) and
pins of their oracle."""
import ctypes

import numpy as np
import pytest

from oracle import decoder as D
from oracle import lora as L
from oracle import moe as MO

null, some = ctypes.c_void_p(0), ctypes.c_void_p(256)


def abi():
    from adapter_lora_amd import _abi
    return _abi


def norm(**kw):
    a = dict(dtype=1, x=some, ldx=64, residual=null, ldr=0, weight=some, eps=1e-6, M=4, K=64,
             residual_out=null, ldro=0, out=some, ldo=64, out8=null, ldo8=0, scale=null)
    a.update(kw)
    return abi().lib.lora_rms_norm(*a.values(), null)


def test_rms_norm_refusals():
    INV, UNS = abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED
    odd = ctypes.c_void_p(264)                                   # 8-byte aligned only
    for bad in [dict(dtype=2), dict(dtype=7), dict(M=-1), dict(K=60), dict(K=0), dict(x=null),
                dict(x=odd), dict(ldx=56), dict(ldx=68), dict(weight=null), dict(weight=odd),
                dict(out=null), dict(out=odd), dict(ldo=8), dict(out8=some, ldo8=64),
                dict(scale=some), dict(out8=some, ldo8=60, scale=some), dict(out8=odd, ldo8=64, scale=some),
                dict(residual_out=some, ldro=64), dict(residual=odd, ldr=64),
                dict(residual=some, ldr=32), dict(residual=some, ldr=64, residual_out=some, ldro=8),
                dict(eps=-1.0), dict(eps=float("nan"))]:
        assert norm(**bad) == INV, bad
    assert norm(K=32776, ldx=32776, ldo=32776) == UNS
    assert norm(M=0, x=null, out=null) == abi().LORA_OK          # nothing to do
    q = abi().lib.lora_quantize_rows
    assert q(1, some, 64, 4, 64, null, 64, some, null) == INV
    assert q(1, some, 64, 4, 64, some, 64, null, null) == INV
    assert q(1, some, 64, 4, 64, some, 32, some, null) == INV
    assert q(2, some, 64, 4, 64, some, 64, some, null) == INV
    assert q(1, some, 64, 4, 65536, some, 64, some, null) == UNS


def table(K=128, dtype=1):
    w = abi().lora_weights_t()
    w.dtype, w.K, w.n_slices, w.L, w.r_max = dtype, K, 1, 4, 16
    w.slice_offsets[0], w.slice_offsets[1] = 0, 128
    w.A = w.B = some
    w.a_off = w.b_off = ctypes.cast(some, ctypes.POINTER(ctypes.c_int64))
    w.rank = ctypes.cast(some, ctypes.POINTER(ctypes.c_int32))
    seg = abi().lora_segments_t()
    for f in ("sorted_idx", "seg_indptr", "req_to_lora", "num_segments", "tile_info",
              "tile_rows", "num_tiles"):
        setattr(seg, f, ctypes.cast(some, ctypes.POINTER(ctypes.c_int32)))
    seg.L, seg.max_tiles = 4, 8
    return w, seg


def test_linear_fp8_refusals():
    INV, UNS = abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED
    odd = ctypes.c_void_p(264)

    def call(w, table_seg, **kw):
        a = dict(W8=some, ldw=128, w_scale=some, x8=some, ldx8=128, x_scale=some, x=some, ldx=128,
                 M=8, seg=ctypes.byref(table_seg), y=some, ldy=128, ws=some, bytes=1 << 20)
        a.update(kw)
        return abi().lib.lora_linear_fp8(ctypes.byref(w), *a.values(), null)

    w, seg = table()
    for bad in [dict(W8=null), dict(W8=odd), dict(ldw=112), dict(ldw=136), dict(w_scale=null),
                dict(x8=null), dict(ldx8=120), dict(x_scale=null), dict(x=null), dict(ldx=64),
                dict(M=-1), dict(M=(1 << 24) + 1), dict(seg=None), dict(y=null), dict(y=odd),
                dict(ldy=120), dict(ws=null), dict(ws=odd), dict(bytes=64)]:
        assert call(w, seg, **bad) == INV, bad
    assert call(w, seg, M=0, x=null) == abi().LORA_OK
    assert call(*table(K=136), ldw=144, ldx8=144, ldx=136) == UNS          # K % 16
    assert call(*table(dtype=0)) == UNS                                    # fp32 table
    # byte offsets past 31 bits: 32 rows of W8 (16 of them would fit), 256 of the
    # larger product, the token rows
    assert call(w, seg, ldw=(1 << 31) // 20 // 16 * 16) == UNS
    assert call(w, seg, M=100, ldw=(1 << 31) // 200 // 16 * 16, bytes=1 << 30) == UNS
    assert call(w, seg, ldx=1 << 28) == UNS and call(w, seg, ldx8=1 << 29) == UNS
    seg.L = 5
    assert call(w, seg) == INV


def experts(**kw):
    e = abi().lora_moe_experts_t()
    a = dict(wdtype=1, E=8, H=64, I=32, topk=2, renormalize=0, router=some, W_gu=some, W_d=some,
             s_gu=null, s_d=null)
    a.update(kw)
    for k, v in a.items():
        setattr(e, k, v)
    return e


def moe_weights(**kw):
    w = abi().lora_moe_weights_t()
    a = dict(dtype=1, L=2, E=8, H=64, I=32, r=16, shared_outer=0, A_gu=some, B_gu=some, A_d=some,
             B_d=some)
    a.update(kw)
    for k, v in a.items():
        setattr(w, k, v)
    w.adapter_enabled = ctypes.cast(some, ctypes.POINTER(ctypes.c_int32))
    return w


def test_moe_decode_refusals():
    lib, INV, UNS = abi().lib, abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED
    odd = ctypes.c_void_p(264)

    def call(ex, w=None, **kw):
        a = dict(ids=some, x=some, ldx=64, M=8, out=some, ldo=64, topk_ids=null, topk_weights=null,
                 ws=some, bytes=1 << 24)
        a.update(kw)
        return lib.lora_moe_decode(ctypes.byref(w) if w else None, ctypes.byref(ex) if ex else None,
                                   *a.values(), null)

    def size(ex, w, M=8):
        return lib.lora_moe_decode_workspace_size(ctypes.byref(w) if w else None, ctypes.byref(ex), M)

    assert call(None) == INV
    for bad in [dict(wdtype=0), dict(E=0), dict(E=257), dict(topk=0), dict(topk=9), dict(H=60),
                dict(I=4), dict(router=null), dict(W_gu=odd), dict(W_d=null), dict(s_gu=some),
                dict(s_d=some), dict(wdtype=2), dict(wdtype=2, s_gu=some),
                dict(wdtype=2, s_gu=some, s_d=some, H=72), dict(E=20, topk=17)]:
        assert call(experts(**bad)) == INV, bad
        assert size(experts(**bad), None) == 0
    for bad in [dict(E=4), dict(H=128), dict(I=64), dict(r=24), dict(L=0), dict(A_gu=null)]:
        assert call(experts(), moe_weights(**bad)) == INV, bad
    assert call(experts(), moe_weights(dtype=0)) == UNS
    for bad in [dict(ids=null), dict(x=null), dict(ldx=56), dict(out=odd), dict(ldo=60), dict(M=-1),
                dict(ws=null), dict(ws=odd), dict(bytes=512)]:
        assert call(experts(), moe_weights(), **bad) == INV, bad
    assert call(experts(), M=65) == UNS
    assert call(experts(), M=0, x=null) == abi().LORA_OK
    assert size(experts(), None, 65) == 0 and size(experts(), None, -1) == 0
    assert size(experts(), moe_weights()) > size(experts(), None) > 0
    # room for the partial sums of every split of a tile but one, fp32 with a tag
    for H, at_least in ((384, 31), (4096, 3), (1024, 15)):
        assert size(experts(H=H, I=320), None, 64) > at_least * 64 * H * 8
    # a workspace serves every smaller batch
    for H in (64, 4096):
        ex = experts(H=H, topk=8)
        sizes = [size(ex, None, m) for m in range(65)]
        assert sizes == sorted(sizes)


def test_binding_refusals():
    import torch
    import adapter_lora_amd as ml
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
    x8, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4)
    with pytest.raises(ml.LoraError, match="out or out8"):
        ml.lora_rms_norm(x, w)
    with pytest.raises(ml.LoraError, match="together"):
        ml.lora_rms_norm(x, w, out8=x8)
    with pytest.raises(ml.LoraError, match="needs a residual"):
        ml.lora_rms_norm(x, w, out=x, residual_out=x)
    with pytest.raises(ml.LoraError, match="vector of 64"):
        ml.lora_rms_norm(x, w.float(), out=x)
    with pytest.raises(ml.LoraError, match="vector of 64"):
        ml.lora_rms_norm(x, torch.ones(72, dtype=bf), out=x)
    with pytest.raises(ml.LoraError, match="shape"):
        ml.lora_rms_norm(x, w, out=torch.zeros(4, 72, dtype=bf))
    with pytest.raises(ml.LoraError, match="unsupported dtype"):
        ml.lora_rms_norm(x.half(), w.half(), out=x.half())
    with pytest.raises(ml.LoraError, match="GPU"):
        ml.lora_rms_norm(x, w, out=x)
    with pytest.raises(ml.LoraError, match="float8"):
        ml.lora_quantize_rows(x, x, s)
    with pytest.raises(ml.LoraError, match="GPU"):
        ml.lora_quantize_rows(x, x8, s)
    tb = type("T", (), dict(dtype=bf, K=64, N=32, L=4, cols=16))()
    W8 = torch.zeros(32, 64, dtype=torch.float8_e4m3fn)
    y = torch.zeros(4, 32, dtype=bf)
    with pytest.raises(ml.LoraError, match="float8"):
        ml.lora_linear_fp8(tb, W8.float(), s, x8, s, x, None, y, None)
    with pytest.raises(ml.LoraError, match="rows"):
        ml.lora_linear_fp8(tb, W8, s, x8[:3], s, x, None, y, None)
    with pytest.raises(ml.LoraError, match="columns"):
        ml.lora_linear_fp8(tb, W8[:, :48], s, x8, s, x, None, y, None)
    with pytest.raises(ml.LoraError, match="one row per output"):
        ml.lora_linear_fp8(tb, W8[:24], s, x8, s, x, None, y, None)
    with pytest.raises(ml.LoraError, match="GPU"):
        ml.lora_linear_fp8(tb, W8, s, x8, s, x, None, y, None)
    z = lambda *shape, dtype=bf: torch.zeros(*shape, dtype=dtype)      # noqa: E731
    for args, kw, match in [
            ((z(8, 64), z(8, 64, 64), z(8, 64, 40), 2), {}, "inconsistent"),
            ((z(8, 64), z(8, 64, 64).float(), z(8, 64, 32).float(), 2), {}, "bfloat16 or"),
            ((z(8, 64).float(), z(8, 64, 64), z(8, 64, 32), 2), {}, "router"),
            ((z(8, 64), z(8, 64, 64), z(8, 64, 32), 2), dict(s_gu=z(8, 64)), "8 bits"),
            ((z(8, 64), z(8, 64, 64, dtype=ml.E4M3), z(8, 64, 32, dtype=ml.E4M3), 2), {}, "8 bits"),
            ((z(8, 64), z(8, 64, 64), z(8, 64, 32), 2), {}, "GPU")]:
        with pytest.raises(ml.LoraError, match=match):
            ml.MoeExperts(*args, **kw)
    ex = type("X", (), dict(H=64, topk=2, ref=None))()
    with pytest.raises(ml.LoraError, match="weights are"):
        ml.lora_moe_decode(None, ex, None, x.float(), x, None)
    with pytest.raises(ml.LoraError, match="columns"):
        ml.lora_moe_decode(None, ex, None, x[:, :56], x, None)
    with pytest.raises(ml.LoraError, match="rows"):
        ml.lora_moe_decode(None, ex, None, x, x[:2], None)
    with pytest.raises(ml.LoraError, match="GPU"):
        ml.lora_moe_decode(None, ex, None, x, x, None)


# ------------------------------------------------------------------ oracle pins
def test_oracle_linear_agrees_with_the_dense_oracle():
    rng = np.random.default_rng(0)
    M, K, sizes, ranks = 9, 32, [16, 8], [4, 0, 8]
    N = sum(sizes)
    x8, W8 = rng.integers(-8, 9, (M, K)) / 4.0, rng.integers(-8, 9, (N, K)) / 4.0
    xs, ws = rng.random(M) + 0.5, rng.random(N) + 0.5
    x = rng.standard_normal((M, K))
    A = [rng.standard_normal((2 * r, K)) for r in ranks]
    B = [rng.standard_normal((N, r)) for r in ranks]
    ids = np.array([0, 2, -1, 1, 0, 2, 2, -1, 0])
    base = (x8 * xs[:, None]) @ (W8 * ws[:, None]).T
    want = L.lora_linear(x, ids, A, B, ranks, sizes, base)
    got, mag, dmag = D.linear_fp8_mag(x8, xs, W8, ws, x, ids, A, B, ranks, sizes)
    assert np.allclose(got, want, rtol=0, atol=1e-12) and (mag + dmag >= np.abs(got) - 1e-12).all()
    assert not dmag[[2, 3, 7]].any()                             # no adapter, an empty slot


@pytest.mark.parametrize("shared", [False, True])
def test_oracle_moe_layer_agrees_with_the_staged_oracle(shared):
    """The whole layer equals base products, gate/up delta, activation, down
    delta and top-k reduce run one after the other."""
    rng = np.random.default_rng(1)
    M, E, k, H, I, Ld, r = 7, 4, 2, 16, 8, 2, 3
    x, router = rng.standard_normal((M, H)), rng.standard_normal((E, H))
    W_gu, W_d = rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    eo = 1 if shared else E
    A_gu, B_gu = rng.standard_normal((Ld, eo, r, H)), rng.standard_normal((Ld, E, 2 * I, r))
    A_d, B_d = rng.standard_normal((Ld, E, r, I)), rng.standard_normal((Ld, eo, H, r))
    tok = np.array([0, 1, -1, 1, 0, 0, -1])
    ids, w = D.route(x, router, k, True)
    assert np.allclose(w.sum(1), 1)
    on = [1, 1]
    c1 = np.stack([W_gu[e] @ x[m] for m in range(M) for e in ids[m]])
    kw = dict(shared_outer=True) if shared else {}
    c1 = MO.moe_gate_up_add(x, c1, ids, tok, on, A_gu, B_gu, **kw)
    c2 = MO.silu_and_mul(c1)
    c3 = np.stack([W_d[e] @ c2[m * k + j] for m in range(M) for j, e in enumerate(ids[m])])
    c3 = MO.moe_down_add(c2, c3, ids, tok, on, A_d, B_d, **kw)
    want = MO.topk_reduce(c3, w)
    got, bound = D.moe_layer_mag(x, ids, w, W_gu, W_d, tok, [A_gu, B_gu, A_d, B_d], on, 2.0 ** -8,
                                 1e-6)
    assert np.allclose(got, want, rtol=0, atol=1e-10) and (bound > 0).all()


def test_oracle_norm_and_route_by_hand():
    x, res = np.array([[1.0, 2.0, 2.0, -4.0]]), np.array([[2.0, 2.0, -2.0, 8.0]])
    h, v = D.rms_norm(x, np.array([1.0, 1.0, 2.0, 0.5]), 0.0, res)
    rms = np.sqrt((9 + 16 + 0 + 16) / 4)
    assert np.array_equal(h, [[3, 4, 0, 4]]) and np.allclose(v, np.array([[3, 4, 0, 2]]) / rms)
    assert np.allclose(D.row_scale(np.array([[0.0, 0.0], [-896.0, 1.0], [1e-60, 0]])),
                       [1.0, 2.0, 2.0 ** -126])
    ids, w = D.route(np.eye(2), np.array([[1.0, 0], [2.0, 3.0], [2.0, 3.0]]), 2, False)
    assert ids.tolist() == [[1, 2], [1, 2]]
    e = np.exp([1.0, 2.0, 2.0])
    assert np.allclose(w[0], e[1:] / e.sum())
