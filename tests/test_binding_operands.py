"""Operands that the binding has to refuse before a launch: rows that overlap
(broadcast or strided by less than their width).  Tensors in host memory stand
in for device ones, so nothing here needs a GPU."""
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


@pytest.mark.parametrize("i", range(3))
def test_overlapping_rows_are_refused(i):
    M, K, N = 4, 64, 64
    x, w, x8, s = z(M, K), z(K), z(M, K, dtype=E4M3), z(M, dtype=torch.float32)
    bad, bad8 = overlapping(M, K)[i], overlapping(M, K, torch.uint8)[i].view(E4M3).as_subclass(OnGpu)
    tb = type("T", (), dict(dtype=BF, K=K, N=N, L=4, cols=16, ref=None))()
    seg = type("S", (), dict(L=4, sorted_idx=z(M, dtype=torch.int32), ref=None))()
    ws = type("W", (), dict(ptr=0, nbytes=0))()
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
        assert ml._matrix(t, "x", t.shape, torch.float32)[1] == ld
        assert ml._rows(t, "x") == ld
