"""lora_linear_int8 in every form that a rule on sizes chooses, at the sizes that reach
it: the lists of test_gpu_decoder_paths.py and test_gpu_ring_tiles.py with 8-bit integers.
Tolerances are those of test_gpu_int8.py."""
import pytest
import torch

from tests import test_gpu_decoder_paths as paths
from tests import test_gpu_ring_tiles as ring
from tests.linear_forms import EVERY_FORM, form
from tests.test_gpu_int8 import Case

SIZES = {**paths.FORMS, **{"large_" + k: v for k, v in paths.LARGE.items()}}


def case_form(case):
    M, K, sizes, ranks = case[:4]
    return form(M, K, sizes, len(ranks))


def test_sizes_reach_every_form():
    reached = {case_form(c) for c in SIZES.values()}
    tiles = [n for n, c in ring.CASES.items() if case_form(c) == ("tiles",)]
    assert set(ring.CASES) - set(tiles) <= {"many_slots"} and reached | {("tiles",)} == EVERY_FORM
    assert {case_form(c) for n, c in SIZES.items() if n.startswith("large_")} == {("units", 128, 256)}
    assert all(case_form(c)[2] == 2 for n, c in SIZES.items() if n.startswith("wide_"))
    assert all(case_form(c) == ("groups", 2) for n, c in SIZES.items() if n.startswith("groups_wide"))


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SIZES))
def test_every_form_matches_oracle(name):
    M, K, sizes, ranks = SIZES[name]
    print(name, case_form(SIZES[name]), flush=True)
    c = Case(M, K, sizes, ranks, None, seed=len(name))
    y = c.run()
    c.check(y)
    torch.cuda.synchronize()
    assert torch.equal(y, c.run())


@pytest.mark.gpu
def test_large_units_integers_bit_exact(monkeypatch):
    monkeypatch.setattr(paths, "Case", Case)
    paths.test_large_units_integers_bit_exact()


@pytest.mark.gpu
def test_large_units_adapters_infinities_stay_with_its_tokens(monkeypatch):
    monkeypatch.setattr(paths, "Case", Case)
    paths.test_large_units_adapters_infinities_stay_with_its_tokens()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,sizes,L", [(40, 272, [8200], 48), (64, 8208, [72], 40), (129, 2064, [2056], 48),
                                         (260, 272, [264, 72], 63), (450, 1040, [15688, 72], 50)])
def test_infinities_of_a_late_slot_stay_with_its_tokens(monkeypatch, M, K, sizes, L):
    monkeypatch.setattr(paths, "Case", Case)
    if M > L:                                          # every slot has tokens
        paths.test_infinities_of_a_late_slot_stay_with_its_tokens(M, K, sizes, L)
        return
    c = Case(M, K, sizes, [16, 32] * (L // 2), list(range(M)), seed=L)
    clean = c.run()
    c.check(clean)
    import adapter_lora_amd as ml
    c.B[35][3, 1] = float("inf")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    y = c.run()
    assert not torch.isfinite(y[35, 3]) and torch.equal(y[:35], clean[:35]) and torch.equal(y[36:], clean[36:])
