"""Forms of the 8-bit decoder-layer calls that a rule on sizes chooses, each at
a size that makes it the chosen one.  Tolerances are those of the files that
Case and Layer come from."""
import pytest
import torch

from tests.test_gpu_linear_fp8 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,sizes,L", [(260, 272, [264, 72], 48), (260, 272, [264, 72], 63), (130, 528, [40], 40),
                                         (300, 144, [13320], 50)])
def test_infinities_of_a_late_slot_stay_with_its_tokens(M, K, sizes, L):
    """Past 64 tokens, with tables of up to 63 slots: an infinite and a NaN value
    in the B of an adapter whose slot and whose segment are 32 or more."""
    import adapter_lora_amd as ml
    g = torch.Generator().manual_seed(L)
    ids = (torch.arange(M)[torch.randperm(M, generator=g)] % (L + 1) - 1).tolist()
    c = Case(M, K, sizes, [16, 32] * (L // 2) + [64] * (L % 2), ids, seed=L)
    clean = c.run()
    c.check(clean)
    order = c.seg.req_to_lora[:int(c.seg.num_segments.item())].tolist()
    assert len(order) == L
    late = [i for i in order[32:] if i >= 32]
    i = late[-1]
    c.B[i][3, 1] = float("inf")
    c.B[i][sum(sizes) - 1, 0] = float("nan")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    y = c.run()
    other = c.ids != i
    assert torch.equal(y[other], clean[other])
    hit = [3, c.N - 1]
    assert not torch.isfinite(y[~other][:, hit]).any()
    rest = [n for n in range(c.N) if n not in hit]
    assert torch.equal(y[~other][:, rest], clean[~other][:, rest])
    assert ml.lora_read_device_error(c.ws_buf.buf) == 0
