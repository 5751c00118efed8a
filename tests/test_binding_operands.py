"""Operands that the binding has to refuse before a launch: rows that overlap
(broadcast or strided by less than their width), and operands on another device
than the call.  Tensors in host memory stand in for device ones, so nothing here
needs a GPU."""
import pytest
import torch

import adapter_lora_amd as ml

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class OnGpu(torch.Tensor):
    """A host tensor that says it lives on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def dev(t):
    return t.as_subclass(OnGpu)


def z(*shape, dtype=BF):
    return dev(torch.zeros(*shape, dtype=dtype))


def overlapping(M, K, dtype=BF):
    """[M, K] operands whose rows start less than K values apart."""
    flat = torch.zeros(M * K, dtype=dtype)
    return [dev(flat[:K].expand(M, K)), dev(flat.as_strided((M, K), (8, 1))), dev(flat.as_strided((M, K), (K - 8, 1)))]


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    """Every library call that a refusal should have come before fails."""
    def launched(*args):
        pytest.fail("the call reached the library")
    for name in ("lora_rms_norm", "lora_quantize_rows", "lora_linear_fp8", "lora_moe_decode", "lora_moe_silu_and_mul",
                 "lora_moe_topk_reduce"):
        monkeypatch.setattr(ml.lib, name, launched)
    monkeypatch.setattr(ml, "stream_handle", lambda stream=None: 0)
    monkeypatch.setattr(ml, "_cur_device", lambda: 0)
    monkeypatch.setattr(ml, "_raw_stream", lambda device: 0)


@pytest.mark.parametrize("i", range(3))
def test_overlapping_rows_are_refused(i):
    M, K, N = 4, 64, 64
    x, w, x8, s = z(M, K), z(K), z(M, K, dtype=E4M3), z(M, dtype=torch.float32)
    bad, bad8 = overlapping(M, K)[i], overlapping(M, K, torch.uint8)[i].view(E4M3).as_subclass(OnGpu)
    tb = type("T", (), dict(dtype=BF, K=K, N=N, L=4, cols=16, ref=None))()
    seg = type("S", (), dict(L=4, sorted_idx=z(M, dtype=torch.int32), ref=None))()
    ws = type("W", (), dict(ptr=0, nbytes=0, buf=z(8)))()
    W8, sn, y = z(N, K, dtype=E4M3), z(N, dtype=torch.float32), z(M, N)
    ex = type("X", (), dict(H=K, topk=2, ref=None))()
    calls = [lambda: ml.lora_rms_norm(bad, w, out=x),
             lambda: ml.lora_rms_norm(x, w, residual=bad, out=x),
             lambda: ml.lora_rms_norm(x, w, residual=x, residual_out=bad, out=x),
             lambda: ml.lora_rms_norm(x, w, out=bad),
             lambda: ml.lora_rms_norm(x, w, out8=bad8, scale=s),
             lambda: ml.lora_quantize_rows(bad, x8, s),
             lambda: ml.lora_quantize_rows(x, bad8, s)]
    bad_w = overlapping(N, K, torch.uint8)[i].view(E4M3).as_subclass(OnGpu)
    for k, v in dict(W8=bad_w, x8=bad8, x=bad, y=bad).items():
        a = dict(table=tb, W8=W8, w_scale=sn, x8=x8, x_scale=s, x=x, seg=seg, y=y, ws=ws)
        a[k] = v
        calls.append(lambda a=a: ml.lora_linear_fp8(**a))
    calls += [lambda: ml.lora_moe_decode(None, ex, None, bad, x, ws),
              lambda: ml.lora_moe_decode(None, ex, None, x, bad, ws),
              # calls that share the older check of rows
              lambda: ml.lora_moe_silu_and_mul(bad, z(M, K // 2)),
              lambda: ml.lora_moe_silu_and_mul(x, overlapping(M, K // 2)[i])]
    for n, call in enumerate(calls):
        with pytest.raises(ml.LoraError, match="overlap"):
            call()
            pytest.fail(f"call {n} was accepted")


def test_rows_that_do_not_overlap_keep_their_stride():
    one = dev(torch.zeros(64).as_strided((1, 64), (3, 1)))       # a single row has no next one
    none = dev(torch.zeros(64).as_strided((0, 64), (3, 1)))
    wide = dev(torch.zeros(4, 96)[:, 16:80])
    for t, ld in ((one, 64), (none, 64), (wide, 96)):
        assert ml._matrix(t, "x", t.shape, torch.float32, 0)[1] == ld
        assert ml._rows(t, "x") == ld


class OnOther(OnGpu):
    """A host tensor that says it lives on device 1."""
    def get_device(self):
        return 1


def calls_of(op):
    """The call with its operands by name, and the names that are tensors or hold them."""
    M, K, N = 4, 64, 64
    x, x8, s = z(M, K), z(M, K, dtype=E4M3), z(M, dtype=torch.float32)
    ws = lambda t: type("W", (), dict(ptr=0, nbytes=0, buf=t))()                                 # noqa: E731
    if op == "norm":
        return ml.lora_rms_norm, dict(x=x, weight=z(K), residual=x, residual_out=z(M, K), out=z(M, K), out8=x8, scale=s)
    if op == "quantize":
        return ml.lora_quantize_rows, dict(x=x, out8=x8, scale=s)
    if op == "linear":
        tb = lambda t: type("T", (), dict(dtype=BF, K=K, N=N, L=4, cols=16, ref=None, A_table=t))()  # noqa: E731
        seg = lambda t: type("S", (), dict(L=4, sorted_idx=t, ref=None))()                      # noqa: E731
        return ml.lora_linear_fp8, dict(table=(tb, z(8)), W8=z(N, K, dtype=E4M3), w_scale=z(N, dtype=torch.float32),
                                        x8=x8, x_scale=s, x=x, seg=(seg, z(M, dtype=torch.int32)), y=z(M, N),
                                        ws=(ws, z(8)))
    ex = lambda t: type("X", (), dict(H=K, topk=2, ref=None, router=t))()                       # noqa: E731
    w = lambda t: type("M", (), dict(c=ml.lora_moe_weights_t(), A_gu=t))()                      # noqa: E731
    return ml.lora_moe_decode, dict(w=(w, z(8)), experts=(ex, z(8)), ids=z(M, dtype=torch.int32), x=x, out=z(M, K),
                                    ws=(ws, z(8)), topk_ids=z(M, 2, dtype=torch.int32),
                                    topk_weights=z(M, 2, dtype=torch.float32))


@pytest.mark.parametrize("op", ["norm", "quantize", "linear", "moe"])
def test_operands_of_another_device_are_refused(op, monkeypatch):
    call, args = calls_of(op)
    real = lambda a: {k: v[0](v[1]) if isinstance(v, tuple) else v for k, v in a.items()}       # noqa: E731
    reached = []
    monkeypatch.setattr(ml.lib, call.__name__, lambda *a: reached.append(a) or 0)
    call(**real(args))
    assert len(reached) == 1                                     # one device: the call goes through
    for k, v in args.items():
        holder = isinstance(v, tuple)
        for t in ((v[1] if holder else v).as_subclass(OnOther), (v[1] if holder else v).as_subclass(torch.Tensor)):
            with pytest.raises(ml.LoraError, match="device|GPU"):
                call(**real(dict(args, **{k: (v[0], t) if holder else t})))
    # all together on a device that is not the call's
    other = {k: (v[0], v[1].as_subclass(OnOther)) if isinstance(v, tuple) else v.as_subclass(OnOther)
             for k, v in args.items()}
    with pytest.raises(ml.LoraError, match="stream on device 0"):
        call(**real(other))
    stream = type("St", (), dict(device_index=1, cuda_stream=0))()
    with pytest.raises(ml.LoraError, match="stream on device 1"):
        call(**real(args), stream=stream)
    assert len(reached) == 1
    call(**real(other), stream=stream)
    assert len(reached) == 2


def test_moe_adapters_of_mixed_types_places_or_a_short_mask_are_refused():
    L, E, r, H, I = 3, 4, 16, 64, 32
    shapes = [(L, E, r, H), (L, E, 2 * I, r), (L, E, r, I), (L, E, H, r)]
    good = [z(*s) for s in shapes] + [z(L, dtype=torch.int32)]
    w = ml.MoeWeights(*good)
    assert (w.L, w.E, w.r, w.H, w.I, w.shared_outer) == (L, E, r, H, I, False)
    for i in range(5):
        for t in (good[i].as_subclass(OnOther), good[i].as_subclass(torch.Tensor)):
            with pytest.raises(ml.LoraError, match="device|GPU"):
                ml.MoeWeights(*good[:i], t, *good[i + 1:])
    for i in range(4):
        with pytest.raises(ml.LoraError, match="one type"):
            ml.MoeWeights(*good[:i], good[i].float(), *good[i + 1:])
    with pytest.raises(ml.LoraError, match="adapter_enabled"):
        ml.MoeWeights(*good[:4], z(L - 1, dtype=torch.int32))
    with pytest.raises(ml.LoraError, match="inconsistent"):
        ml.MoeWeights(good[0], z(L, E, 2 * I + 1, r), *good[2:])
