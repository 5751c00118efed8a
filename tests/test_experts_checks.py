"""Refusals of the experts' products and of the 8-bit integer calls (before any
launch, no GPU), and pins of their oracle."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import adapter_lora_amd as ml
from oracle import decoder as D
from oracle import experts as X
from tests.test_binding_operands import OnGpu, dev, overlapping, z
from tests.test_decoder_checks import abi, null, some, table

odd = ctypes.c_void_p(264)                                       # 8-byte aligned only
BF, E4M3, I8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.float32, torch.int32


# ---------------------------------------------------------------- the library's checks
def test_moe_group_refusals():
    lib, INV = abi().lib, abi().LORA_INVALID_ARG

    def call(**kw):
        a = dict(ids=some, M=4, topk=2, E=8, pairs=some, offsets=some)
        a.update(kw)
        return lib.lora_moe_group(*a.values(), null)

    for bad in [dict(ids=null), dict(M=-1), dict(topk=0), dict(topk=17), dict(E=0), dict(E=257),
                dict(pairs=null), dict(offsets=null), dict(M=1 << 23, topk=3), dict(M=0, offsets=null)]:
        assert call(**bad) == INV, bad


def moe_linear(**kw):
    a = dict(wdtype=1, W=some, w_scale=null, E=8, N=64, K=64, pairs=some, offsets=some, x=some, ldx=64,
             x_scale=null, M=4, topk=2, pair_rows=0, y=some, ldy=64)
    a.update(kw)
    return abi().lib.lora_moe_linear(*a.values(), null)


def test_moe_linear_refusals():
    INV, UNS = abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED
    for bad in [dict(wdtype=0), dict(wdtype=4), dict(W=null), dict(W=odd), dict(E=0), dict(E=257), dict(N=0),
                dict(N=60), dict(K=0), dict(K=60), dict(pairs=null), dict(offsets=null), dict(x=null),
                dict(x=odd), dict(ldx=56), dict(ldx=68), dict(M=-1), dict(topk=0), dict(topk=17), dict(y=null),
                dict(y=odd), dict(ldy=56), dict(ldy=68), dict(M=1 << 24), dict(w_scale=some), dict(x_scale=some)]:
        assert moe_linear(**bad) == INV, bad
    for wdtype in (2, 3):
        eight = dict(wdtype=wdtype, w_scale=some, x_scale=some)
        for bad in [dict(w_scale=null), dict(x_scale=null), dict(K=72, ldx=80), dict(ldx=72), dict(x=odd)]:
            assert moe_linear(**{**eight, **bad}) == INV, bad
    assert moe_linear(K=131072, ldx=131072) == UNS
    assert moe_linear(M=1 << 20, topk=16, N=1 << 16, ldy=1 << 16) == UNS         # more units than a grid holds
    assert moe_linear(M=0, x=null, y=null, pairs=null) == abi().LORA_OK          # nothing to do


def test_int8_rows_refusals():
    INV, UNS = abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED

    def norm(**kw):
        a = dict(dtype=1, x=some, ldx=64, residual=null, ldr=0, weight=some, eps=1e-6, M=4, K=64,
                 residual_out=null, ldro=0, out=some, ldo=64, out8=some, ldo8=64, scale=some)
        a.update(kw)
        return abi().lib.lora_rms_norm_int8(*a.values(), null)

    for bad in [dict(dtype=3), dict(M=-1), dict(K=60), dict(x=null), dict(x=odd), dict(ldx=56), dict(weight=null),
                dict(out=odd), dict(ldo8=60), dict(out8=odd), dict(scale=null), dict(out8=null, scale=null),
                dict(out8=null), dict(residual_out=some, ldro=64), dict(eps=-1.0), dict(eps=float("nan"))]:
        assert norm(**bad) == INV, bad
    assert norm(K=32776, ldx=32776, ldo=32776, ldo8=32776) == UNS
    assert norm(M=0, x=null) == abi().LORA_OK
    q = abi().lib.lora_quantize_rows_int8
    assert q(1, some, 64, 4, 64, null, 64, some, null) == INV
    assert q(1, some, 64, 4, 64, some, 64, null, null) == INV
    assert q(1, some, 64, 4, 64, some, 32, some, null) == INV
    assert q(3, some, 64, 4, 64, some, 64, some, null) == INV
    assert q(1, some, 64, 4, 65536, some, 64, some, null) == UNS


def test_linear_int8_refusals():
    INV, UNS = abi().LORA_INVALID_ARG, abi().LORA_UNSUPPORTED

    def call(w, table_seg, **kw):
        a = dict(W8=some, ldw=128, w_scale=some, x8=some, ldx8=128, x_scale=some, x=some, ldx=128,
                 M=8, seg=ctypes.byref(table_seg), y=some, ldy=128, ws=some, bytes=1 << 20)
        a.update(kw)
        return abi().lib.lora_linear_int8(ctypes.byref(w), *a.values(), null)

    w, seg = table()
    for bad in [dict(W8=null), dict(W8=odd), dict(ldw=112), dict(ldw=136), dict(w_scale=null), dict(x8=null),
                dict(ldx8=120), dict(x_scale=null), dict(x=null), dict(ldx=64), dict(M=-1), dict(seg=None),
                dict(y=null), dict(y=odd), dict(ldy=120), dict(ws=null), dict(ws=odd), dict(bytes=64)]:
        assert call(w, seg, **bad) == INV, bad
    assert call(w, seg, M=0, x=null) == abi().LORA_OK
    assert call(*table(K=136), ldw=144, ldx8=144, ldx=136) == UNS          # K % 16
    assert call(*table(dtype=0)) == UNS                                    # fp32 table
    # a sum of K products of -128 by -128 has to stay below 2^31
    assert call(*table(K=131072), ldw=131072, ldx8=131072, ldx=131072, bytes=1 << 30) == UNS
    assert call(w, seg, ldx=1 << 28) == UNS and call(w, seg, ldx8=1 << 29) == UNS


# ---------------------------------------------------------------- the binding's checks
@pytest.fixture
def no_launch(monkeypatch):
    def launched(*args):
        pytest.fail("the call reached the library")
    for name in ("lora_rms_norm", "lora_rms_norm_int8", "lora_quantize_rows", "lora_quantize_rows_int8",
                 "lora_linear_int8", "lora_moe_group", "lora_moe_linear"):
        monkeypatch.setattr(ml.lib, name, launched)
    monkeypatch.setattr(ml, "stream_handle", lambda stream=None: 0)
    monkeypatch.setattr(ml, "_cur_device", lambda: 0)
    monkeypatch.setattr(ml, "_raw_stream", lambda device: 0)


def made(E=4, P=8, topk=2):
    g = ml.MoeGroups(P, E, device="cpu")
    g.device, g.count, g.topk = 0, P, topk
    return g


class Elsewhere(OnGpu):
    def get_device(self):
        return 1


def test_binding_refusals_moe(no_launch):
    g, W, x, y = made(), z(4, 16, 32), z(4, 32), z(8, 16)
    W8, x8 = z(4, 16, 32, dtype=I8), z(4, 32, dtype=I8)
    sw, sx = z(4, 16, dtype=F32), z(4, dtype=F32)

    def call(W=W, x=x, topk=2, groups=g, y=y, **kw):
        return lambda: ml.lora_moe_linear(W, x, topk, groups, y, **kw)

    bad = [call(W=z(4, 16, 32, dtype=F32)), call(W=z(16, 32)), call(W=z(5, 16, 32)), call(x=z(4, 24)),
           call(x=z(5, 32)), call(x=z(4, 32, dtype=F32)), call(x=x8), call(y=z(8, 24)), call(y=z(6, 16)),
           call(y=z(8, 16, dtype=F32)), call(topk=4), call(topk=0), call(w_scale=sw), call(x_scale=sx),
           call(W=W8, x=x8), call(W=W8, x=x8, w_scale=sw), call(W=W8, x=x8, x_scale=sx),
           call(W=W8, x=x8, w_scale=z(4, 8, dtype=F32), x_scale=sx), call(W=W8, x=x8, w_scale=sw, x_scale=z(3, dtype=F32)),
           call(W=W8, x=x, w_scale=sw, x_scale=sx), call(groups=made(P=6)), call(groups=made(E=3)),
           call(groups=made(P=8, topk=1)), call(W=z(4, 32, 16).transpose(1, 2)),
           call(y=torch.zeros(8, 16, dtype=BF)), call(x=torch.zeros(4, 32, dtype=BF)),
           call(W=torch.zeros(4, 16, 32, dtype=BF).as_subclass(Elsewhere)),
           call(y=torch.zeros(8, 16, dtype=BF).as_subclass(Elsewhere))]
    bad += [call(x=o) for o in overlapping(4, 32)] + [call(y=o) for o in overlapping(8, 16)[:2]]
    ids = z(4, 2, dtype=I32)
    bad += [lambda: ml.lora_moe_group(z(4, 2, dtype=torch.int64), g), lambda: ml.lora_moe_group(z(8, dtype=I32), g),
            lambda: ml.lora_moe_group(z(5, 2, dtype=I32), g), lambda: ml.lora_moe_group(z(2, 4, dtype=I32).t(), g),
            lambda: ml.lora_moe_group(torch.zeros(4, 2, dtype=I32), g),
            lambda: ml.lora_moe_group(ids.as_subclass(Elsewhere), g),
            lambda: ml.MoeGroups(8, 0, device="cpu"), lambda: ml.MoeGroups(8, 257, device="cpu")]
    for f in bad:
        with pytest.raises(ml.LoraError):
            f()


def test_binding_refusals_int8(no_launch):
    x, w, x8, s = z(4, 64), z(64), z(4, 64, dtype=I8), z(4, dtype=F32)
    for f in [lambda: ml.lora_quantize_rows(x, z(4, 64, dtype=torch.uint8), s),
              lambda: ml.lora_quantize_rows(x, z(4, 56, dtype=I8), s),
              lambda: ml.lora_quantize_rows(x, x8, z(3, dtype=F32)),
              lambda: ml.lora_quantize_rows(x, x8, z(4)),
              lambda: ml.lora_quantize_rows(x, torch.zeros(4, 64, dtype=I8), s),
              lambda: ml.lora_rms_norm(x, w, out8=x8),
              lambda: ml.lora_rms_norm(x, w, out8=z(4, 64, dtype=torch.uint8), scale=s)]:
        with pytest.raises(ml.LoraError):
            f()
    for o in overlapping(4, 64, torch.int8):
        with pytest.raises(ml.LoraError):
            ml.lora_quantize_rows(x, o, s)
    tb = type("T", (), dict(dtype=BF, K=64, N=64, L=4, cols=16, ref=None, A_table=z(8)))()
    seg = type("S", (), dict(L=4, sorted_idx=z(4, dtype=I32), ref=None))()
    ws = type("W", (), dict(ptr=0, nbytes=0, buf=z(8)))()
    W8, sn, y = z(64, 64, dtype=I8), z(64, dtype=F32), z(4, 64)
    e8 = z(4, 64, dtype=torch.uint8).view(E4M3)
    for a in [(W8, sn, e8, s, x, y), (z(64, 64, dtype=torch.uint8).view(E4M3), sn, x8, s, x, y), (W8, sn, x8, z(3, dtype=F32), x, y),
              (W8, z(63, dtype=F32), x8, s, x, y), (W8, sn, x8, s, z(4, 64, dtype=F32), y), (W8, sn, x8, s, x, z(5, 64))]:
        W8_, sn_, x8_, s_, x_, y_ = a
        with pytest.raises(ml.LoraError):
            ml.lora_linear_int8(tb, W8_, sn_, x8_, s_, x_, seg, y_, ws)


def test_quantize_rows_without_an_output(monkeypatch):
    """Refused by the library, as a LoraError, not by an attribute of None."""
    monkeypatch.setattr(ml, "_cur_device", lambda: 0)
    monkeypatch.setattr(ml, "_raw_stream", lambda device: 0)
    with pytest.raises(ml.LoraError):
        ml.lora_quantize_rows(z(4, 64), None, z(4, dtype=F32))


# ---------------------------------------------------------------- pins of the oracle
def test_group_pins():
    pairs, offsets = X.group([[2, 0], [5, 2], [-1, 0], [2, 9]], 6)
    assert pairs.tolist() == [1, 5, 0, 3, 6, 2, 4, 7] and offsets.tolist() == [0, 2, 2, 5, 5, 5, 6]
    pairs, offsets = X.group(np.zeros((0, 2)), 3)
    assert pairs.size == 0 and offsets.tolist() == [0, 0, 0, 0]
    rng = np.random.default_rng(0)
    ids = rng.integers(-2, 9, (50, 3))
    pairs, offsets = X.group(ids, 7)
    assert sorted(pairs.tolist()) == list(range(150))
    key = np.where((ids.reshape(-1) < 0) | (ids.reshape(-1) >= 7), 7, ids.reshape(-1))
    assert np.array_equal(pairs, np.argsort(key, kind="stable"))     # another way to the same order
    assert offsets.tolist() == [int((key < e).sum()) for e in range(8)]


def test_grouped_linear_pins():
    rng = np.random.default_rng(1)
    M, topk, E, N, K = 5, 2, 4, 3, 6
    ids = rng.integers(-1, E + 1, (M, topk))
    W, x, xp = rng.normal(size=(E, N, K)), rng.normal(size=(M, K)), rng.normal(size=(M * topk, K))
    for rows, pair_rows in ((x, False), (xp, True)):
        y, mag = X.grouped_linear_mag(ids, rows, W, pair_rows)
        for m in range(M):
            for k in range(topk):
                f, e = m * topk + k, ids[m, k]
                if not 0 <= e < E:
                    assert np.isnan(y[f]).all()
                    continue
                want = [sum(W[e, n, j] * rows[f if pair_rows else m, j] for j in range(K)) for n in range(N)]
                assert np.allclose(y[f], want, atol=1e-12) and (mag[f] >= np.abs(y[f]) - 1e-12).all()
    # the pairs' own rows repeated from the tokens': the same
    assert np.allclose(X.grouped_linear_mag(ids, np.repeat(x, topk, 0), W, True)[0],
                       X.grouped_linear_mag(ids, x, W, False)[0], equal_nan=True)
    # scales are those of the rows and of the expert's columns
    sx, sw = rng.uniform(1, 2, M), rng.uniform(1, 2, (E, N))
    y = X.grouped_linear_mag(ids, x, W, False)[0]
    ys = X.grouped_linear_mag(ids, x, W, False, sx, sw)[0]
    e = np.clip(ids.reshape(-1), 0, E - 1)
    assert np.allclose(ys, y * np.repeat(sx, topk)[:, None] * sw[e], equal_nan=True)


def test_quantize_int8_pins():
    v = np.array([[0.0, 0, 0, 0], [127, -63.5, 0.5, 1.5], [254, -1, 1, 3], [1e-44, 0, -1e-44, 0]])
    q, s = X.quantize_int8(v)
    assert s.tolist() == [1.0, 1.0, 2.0, 2.0 ** -126]
    assert q.tolist() == [[0, 0, 0, 0], [127, -64, 0, 2], [127, 0, 0, 2], [0, 0, 0, 0]]
    rng = np.random.default_rng(2)
    v = rng.normal(size=(20, 64)).astype(np.float32).astype(np.float64)
    q, s = X.quantize_int8(v)
    assert np.abs(q).max() == 127 and (np.abs(q * s[:, None] - v) <= 0.5 * s[:, None] * (1 + 1e-12)).all()
    # half of a row's largest value lies next to a tie: the scale's own rounding decides
    top = rng.uniform(1, 2, 400).astype(np.float32).astype(np.float64)
    q, s = X.quantize_int8(np.stack([top, top / 2], 1))
    for q1, t, s1 in zip(q[:, 1], top, s):
        assert q1 == (64 if Fraction(t) >= 127 * Fraction(s1) else 63)
    assert set(q[:, 1]) == {63.0, 64.0}


def test_row_scale_int8_is_not_the_other_formats():
    v = np.array([[448.0, 127.0]])
    assert D.row_scale(v)[0] == 1.0 and X.row_scale_int8(v)[0] == np.float64(np.float32(448 / 127))
