"""Edges of the products in tiles (ring_product.hpp): what the rings held before does not
come back past K, tables of more slots than a wavefront has lanes beside an
adapter's infinities, and the checks of the checked library."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import test_gpu_moe_linear as X
from tests.linear_forms import form
from tests.test_gpu_ring_tiles import KINDS

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG_LIB = os.path.join(ROOT, "adapter_lora_amd", "libmlora_debug.so")

# every class of rows: a tile's rings hold 3 to 6 stages of W with 256 columns, 4 to 6 with 128
COUNTS = [256, 192, 128, 64, 250, 130, 65, 1]


@pytest.mark.parametrize("width", ["half tiles", "whole tiles"])
@pytest.mark.parametrize("stage", range(7))
def test_w_of_an_earlier_stage_does_not_come_back(width, stage):
    """K of seven stages and 16 bytes of an eighth, whose other W values are read past K: an
    infinity of W in any stage before it meets x's zeros there only if the ring still
    holds it, and would turn the column's infinities into NaN."""
    K = 64 * 7 + 8
    E = 8 if width == "half tiles" else 256
    M = sum(COUNTS) if width == "half tiles" else sum(COUNTS) + 200
    c = X.Case("bf16", M, 1, E, 72, K, COUNTS, seed=stage)
    assert X.form("bf16", M, E, 72, K) == width
    c.W[:8, 5, 64 * stage:64 * stage + 8] = float("inf")      # the chunk of the values that are there
    c.W[:8, 70, 64 * stage + 24:64 * stage + 32] = float("-inf")
    c.W[:8, 40, 64 * stage + 56:64 * stage + 64] = float("inf")
    c.x.abs_().clamp_(min=2 ** -6)                            # infinities of one sign only
    want = c.oracle()[0]
    y = c.run()
    got = np.asarray(y.double().cpu())
    on = ~np.isnan(want[:, 0])
    hit = np.array([n in (5, 40, 70) for n in range(72)])
    assert np.isinf(want[on][:, hit]).all() and np.array_equal(got[on][:, hit], want[on][:, hit])
    c.W[:8, [5, 40, 70]] = 0
    clean = c.run()
    assert torch.equal(y[:, torch.tensor(~hit)], clean[:, torch.tensor(~hit)])
    c.check(clean)


@pytest.mark.parametrize("kind", list(KINDS))
def test_infinities_beside_eighty_slots(kind):
    """More slots than lanes, so that segments are looked up in memory, and an infinity in
    the B of a late slot: it stays with its tokens."""
    import adapter_lora_amd as ml
    M, K, N, L = 2000, 1040, 8192, 80
    assert form(M, K, [N], L) == ("tiles",)
    c = KINDS[kind](M, K, [N], [16, 32] * (L // 2), (torch.arange(M) % (L + 1) - 1).tolist(), seed=4)
    clean = c.run()
    c.check(clean)
    for i in (2, 71):
        c.B[i][3, 1] = float("inf")
        c.B[i][N - 1, 0] = float("nan")
    c.table = ml.LoraTable(c.A, c.B, c.ranks, [N], K, torch.bfloat16)
    y = c.run()
    mine = (c.ids == 2) | (c.ids == 71)
    assert mine.any() and not torch.isfinite(y[mine][:, [3, N - 1]]).any()
    y[:, [3, N - 1]] = torch.where(mine[:, None], clean[:, [3, N - 1]], y[:, [3, N - 1]])
    assert torch.equal(y, clean)
    assert ml.lora_read_device_error(c.ws_buf.buf) == 0


def test_checked_library_tables():
    """The projections' tiles and their 8-bit integers on the checked library: valid tables
    raise nothing, a token past the batch is reported and alone lost."""
    assert os.path.exists(DEBUG_LIB), "run __graft_entry__.build() first"
    env = dict(os.environ, MLORA_LIB=DEBUG_LIB)
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "debug_tiles_run.py")], env=env,
                       capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res.pop("lib") == "libmlora_debug.so" and len(res) == 8
    for name, v in res.items():
        assert v["valid_err"] == 0 and v["valid_exact"], (name, v)
        assert v["err"] == 4 and v["padding_untouched"] and v["others_exact"], (name, v)    # LORA_DEVERR_TABLE
