"""Sums over K of products of 8-bit integers are 32-bit integers in every form of
lora_linear_int8 and lora_moe_linear: bit for bit, where the parts of K are past what
24 bits hold and cancel, and at the largest sum that the limit of K allows.

With unit scales the only rounding of a whole-number sum below 2^24 is y's to bf16,
so outputs are compared bit for bit with the exact sums rounded once."""
import pytest
import torch

from tests.linear_forms import EVERY_FORM, form
from tests.test_gpu_int8 import Case
from tests.test_gpu_moe_linear import Case as Experts

BF, I8 = torch.bfloat16, torch.int8
K = 128 * 128 + 16

# M, slice sizes: every form of the projection at this K
SIZES = {
    "one_token": (1, [264]),
    "one_token_wide": (1, [8192, 6152]),
    "twenty": (20, [200, 72]),
    "twenty_wide": (20, [8200]),
    "sixty_four": (64, [264]),
    "sixty_four_wide": (64, [8200]),
    "groups": (130, [72]),
    "groups_wide": (129, [1032, 1024]),
    "units": (300, [2056]),
    "large_units": (300, [13320]),
    "tiles": (512, [28672]),
}


def test_sizes_reach_every_form():
    assert {form(M, K, sizes, 3) for M, sizes in SIZES.values()} == EVERY_FORM


def cancelling(rows, width, g):
    """(x, W) of whole numbers: 64 pairs of blocks of 128 values of K, the second of each
    with W's sign turned, and 16 values that stay.  Sixteen blocks of one sign add up
    to 16 x 128 x 96^2 = 18.9e6 at least, past 2^24."""
    def blocks(n):
        v = torch.randint(96, 128, (n, 64, 1, 128), generator=g, device="cuda", dtype=I8)
        return v.expand(n, 64, 2, 128).clone()
    x, W = blocks(rows), blocks(width)
    W[:, :, 1].neg_()
    def tail(n):
        return torch.randint(-5, 6, (n, 16), generator=g, device="cuda", dtype=I8)
    x, W = (torch.cat([v.reshape(v.shape[0], -1), tail(v.shape[0])], 1) for v in (x, W))
    return x, W


def exact(x, W):
    return x[:, -16:].double() @ W[:, -16:].double().t()


@pytest.mark.gpu
@pytest.mark.parametrize("adapters", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
def test_projection_sums_that_cancel(name, adapters):
    """With adapters of factors in {-1, 0, 1} the deltas are whole numbers too."""
    print(name, adapters, flush=True)
    M, sizes = SIZES[name]
    ids = None if adapters else [-1] * M
    c = Case(M, K, sizes, [16, 0, 64], ids, seed=len(name), integers=True)
    c.x8, c.W8 = cancelling(M, c.N, torch.Generator(device="cuda").manual_seed(M))
    want = exact(c.x8, c.W8)
    for i, r in enumerate(c.ranks):
        on = c.ids == i
        if r and on.any():
            A = c.A[i].double().reshape(len(sizes), r, K)
            S = torch.stack([c.x[on].double() @ a.t() for a in A])
            B = c.B[i].double().split(sizes)
            want[on] += torch.cat([s @ b.t() for s, b in zip(S, B)], 1)
    assert want.abs().max() < 2 ** 24
    got = c.run()
    bad = got != want.float().to(BF)
    assert not bad.any(), (int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("M,sizes", [(1, [8]), (20, [72]), (64, [24, 8]), (70, [8]), (300, [2056]), (512, [28672])])
def test_projection_largest_sums(M, sizes):
    """131056 products of -128 by -128, 2147221504 and 16 KiB below 2^31, beside columns of
    -128 by 127, at the limit of K."""
    Kmax = 131056
    c = Case(M, Kmax, sizes, [0], [-1] * M, seed=1, integers=True)
    c.x8 = torch.full((M, Kmax), -128, dtype=I8, device="cuda")
    c.W8 = torch.full((c.N, Kmax), -128, dtype=I8, device="cuda")
    c.W8[1::2] = 127
    want = torch.tensor([128 * 128 * Kmax, -128 * 127 * Kmax], device="cuda").float().to(BF)
    assert torch.equal(c.run(), want.repeat(c.N // 2).expand(M, c.N))


# M, topk, E, N, pairs of each expert: the streaming form of 16 and 32 rows, tiles of half
# and of all the columns
EXPERTS = {
    "one_token": (1, 2, 8, 264, None),
    "few_32_rows": (64, 2, 8, 24, [30, 2, 33, 1, 31, 0, 16, 15]),
    "half_tiles": (500, 2, 3, 264, [1, 257, 700]),
    "whole_tiles": (900, 1, 40, 1800, [60, 100, 192, 256, 257]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts_sums_that_cancel(name):
    print(name, flush=True)
    M, topk, E, N, counts = EXPERTS[name]
    c = Experts("int8", M, topk, E, 8, 16, counts, seed=len(name), integers=True)
    x, W = cancelling(M, E * N, torch.Generator(device="cuda").manual_seed(M))
    c.x, c.W, c.N, c.K, c.ws = x, W.reshape(E, N, K), N, K, torch.ones(E, N, device="cuda")
    y, ids = c.run(), c.ids.flatten().long()
    token = torch.arange(M, device="cuda").repeat_interleave(topk)
    for e in range(E):
        on = ids == e
        assert torch.equal(y[on], exact(x[token[on]], c.W[e]).float().to(BF))
    assert (y[ids >= E] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,topk,E,N", [(1, 1, 2, 8), (20, 1, 1, 40), (300, 2, 3, 72), (2100, 1, 256, 8)])
def test_experts_largest_sums(M, topk, E, N):
    Kmax = 131056
    c = Experts("int8", M, topk, E, 8, 16, seed=2, integers=True)
    c.x = torch.full((M, Kmax), -128, dtype=I8, device="cuda")
    c.W = torch.full((E, N, Kmax), -128, dtype=I8, device="cuda")
    c.W[:, 1::2] = 127
    c.N, c.K, c.ws = N, Kmax, torch.ones(E, N, device="cuda")
    want = torch.tensor([128 * 128 * Kmax, -128 * 127 * Kmax], device="cuda").float().to(BF)
    assert torch.equal(c.run(), want.repeat(N // 2).expand(M * topk, N))
