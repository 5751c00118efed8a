"""Buffers of the pairs by expert, and operands of the experts' products that the binding
refuses before a launch: nothing here needs a GPU."""
import pytest
import torch

import adapter_lora_amd as ml
from tests.test_binding_operands import z
from tests.test_experts_checks import E4M3, F32, I8, made


@pytest.mark.parametrize("name", ["pairs", "offsets"])
def test_buffers_stay_what_the_calls_know(name):
    """The calls keep the buffers' addresses, so a buffer cannot be replaced by another
    one that they would not see."""
    g = ml.MoeGroups(8, 4, device="cpu")
    kept = getattr(g, name)
    with pytest.raises(AttributeError):
        setattr(g, name, torch.empty(64, dtype=torch.int32))
    assert getattr(g, name) is kept
    assert (g.pairs_ptr, g.offsets_ptr) == (g.pairs.data_ptr(), g.offsets.data_ptr())


def test_construction_writes_nothing(monkeypatch):
    """A fill on the constructing stream could land after another stream's first groups."""
    def filled(*args, **kw):
        pytest.fail("the buffers are filled")
    monkeypatch.setattr(torch, "zeros", filled)
    monkeypatch.setattr(torch, "full", filled)
    g = ml.MoeGroups(8, 4, device="cpu")
    assert g.pairs.shape == (8,) and g.offsets.shape == (5,) and g.count == 0


class Reached(Exception):
    pass


@pytest.fixture
def calls(monkeypatch):
    """The library's calls are only reached."""
    def reached(*args):
        raise Reached
    for name in ("lora_linear_fp8", "lora_linear_int8", "lora_moe_linear", "lora_quantize_rows_int8"):
        monkeypatch.setattr(ml.lib, name, reached)
    monkeypatch.setattr(ml, "_cur_device", lambda: 0)
    monkeypatch.setattr(ml, "_raw_stream", lambda device: 0)


def test_scales_with_others_between_are_refused(calls):
    """One scale a row: scales of groups along K, or rows of a wider matrix, would be read
    as if they were the next rows'.  The front of a longer vector is taken."""
    f = lambda *s: z(*s, dtype=F32)               # noqa: E731
    W, x8, y = z(4, 16, 32, dtype=I8), z(4, 32, dtype=I8), z(8, 16)

    def experts(w_scale, x_scale):
        ml.lora_moe_linear(W, x8, 2, made(), y, w_scale=w_scale, x_scale=x_scale)

    tb = type("T", (), dict(dtype=torch.bfloat16, K=64, N=64, L=4, cols=16, ref=None, A_table=z(8)))()
    seg = type("S", (), dict(L=4, sorted_idx=z(4, dtype=torch.int32), ref=None))()
    ws = type("W", (), dict(ptr=0, nbytes=0, buf=z(8)))()

    def linear(call, dtype, w_scale, x_scale):
        e = lambda *s: z(*s, dtype=torch.uint8).view(dtype)       # noqa: E731
        call(tb, e(64, 64), w_scale, e(4, 64), x_scale, z(4, 64), seg, z(4, 64), ws)

    def rows(scale):
        ml.lora_quantize_rows(z(4, 64), z(4, 64, dtype=I8), scale)

    i8, e4 = (ml.lora_linear_int8, I8), (ml.lora_linear_fp8, E4M3)
    for call in [lambda: experts(f(4, 24), f(4)), lambda: experts(f(4, 16, 2), f(4)), lambda: experts(f(4, 16), f(4, 2)),
                 lambda: linear(*i8, f(64, 2), f(4)), lambda: linear(*i8, f(64), f(4, 2)),
                 lambda: linear(*e4, f(64, 2), f(4)), lambda: linear(*e4, f(64), f(4, 2)), lambda: rows(f(4, 2))]:
        with pytest.raises(ml.LoraError):
            call()
    for call in [lambda: experts(f(4, 16), f(4)), lambda: experts(f(64), f(4, 1)), lambda: experts(f(4, 16, 1), f(9)),
                 lambda: linear(*i8, f(64), f(6, 1)), lambda: linear(*i8, f(1, 64), f(1, 4)),
                 lambda: linear(*e4, f(70), f(4)), lambda: rows(f(9)), lambda: rows(f(9, 1))]:
        with pytest.raises(Reached):
            call()
