"""Run by tests/test_gpu_ring_edges.py in a child process on the library built with
MLORA_DEBUG.  lora_linear_fp8 in its tiles of 256 x 256 and lora_linear_int8 in each
form get a valid segment table and one with a token index past the batch, which names
padding rows of this script's own buffers; the tiles once more with a table of
80 slots and with infinities in B.  Prints one JSON line."""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import adapter_lora_amd as ml  # noqa: E402
from tests import test_gpu_int8, test_gpu_linear_fp8  # noqa: E402
from tests.linear_forms import form  # noqa: E402

PAD = 64


def padded(t, value):
    full = torch.full((t.shape[0] + PAD,) + t.shape[1:], value, device="cuda").to(t.dtype)
    full[:t.shape[0]] = t
    return full[:t.shape[0]], full


def linear(Case, M, K, sizes, ranks=(16, 32), special=False):
    c = Case(M, K, sizes, list(ranks), None, seed=3, integers=True)
    if special:
        c.B[1][3, 1] = float("inf")
        c.table = ml.LoraTable(c.A, c.B, c.ranks, sizes, K, torch.bfloat16)
    c.x, _ = padded(c.x, 7.0)
    c.x8 = padded(c.x8.float(), 7.0)[1].to(c.x8.dtype)[:M]
    c.xs, _ = padded(c.xs, 7.0)
    y, full = padded(torch.zeros(M, c.N, dtype=torch.bfloat16, device="cuda"), 7.0)
    c.run(y)
    torch.cuda.synchronize()
    want = y.clone()
    r = {"valid_err": ml.lora_read_device_error(c.ws_buf.buf), "valid_exact": True}
    if not special:
        o = torch.from_numpy(c.oracle()[0]).cuda()
        small = o.abs() <= 256
        r["valid_exact"] = bool((want[small].double() == o[small]).all() and small.any())
    # a token of segment 1 is named past the batch: it alone is lost
    c.ws_buf = ml.Workspace.for_table(c.table, M)
    pos = int(c.seg.seg_indptr[1].item()) + 2
    lost = int(c.seg.sorted_idx[pos].item())
    c.seg.sorted_idx[pos] = M + 5
    y.zero_()
    c.run(y)
    torch.cuda.synchronize()
    want[lost] = 0
    r.update(err=ml.lora_read_device_error(c.ws_buf.buf), padding_untouched=bool((full[M:].float() == 7).all()),
             others_exact=bool(torch.equal(y.nan_to_num(nan=3e38), want.nan_to_num(nan=3e38))))
    return r


FP8, INT8 = test_gpu_linear_fp8.Case, test_gpu_int8.Case
TILES, SLOTS = (500, 1024, [28672]), (2000, 1024, [8192])
assert form(*TILES, 2) == form(*SLOTS, 80) == ("tiles",)
out = {"lib": os.path.basename(ml._abi.LIB_PATH)}
out["tiles_fp8"] = linear(FP8, *TILES)
out["tiles_fp8_special"] = linear(FP8, *TILES, special=True)
out["tiles_int8"] = linear(INT8, *TILES)
out["tiles_int8_slots"] = linear(INT8, *SLOTS, ranks=[16, 32] * 40)
out["tiles_int8_special_slots"] = linear(INT8, *SLOTS, ranks=[16, 32] * 40, special=True)
out["decode_int8"] = linear(INT8, 40, 256, [72])
out["groups_int8"] = linear(INT8, 150, 2048, [72])
out["units_int8"] = linear(INT8, 150, 256, [264])
print(json.dumps(out), flush=True)
