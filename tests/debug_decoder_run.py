"""Run by tests/test_gpu_decoder_layer.py in a child process on the library
built with MLORA_DEBUG.  lora_linear_fp8 in its three forms gets a valid
segment table and one with a token index past the batch, which names padding
rows of this script's own buffers; lora_moe_decode has no table to corrupt
and runs twice.  With MLORA_DEBUG_WAIT_FAULT=1 every bounded wait misses: the
calls report it and end normally.  Prints one JSON line."""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import adapter_lora_amd as ml  # noqa: E402
from tests.test_gpu_linear_fp8 import Case, F64  # noqa: E402
from tests.test_gpu_moe_decode import Layer  # noqa: E402

PAD = 64
out = {"lib": os.path.basename(ml._abi.LIB_PATH)}


def padded(t, value):
    full = torch.full((t.shape[0] + PAD,) + t.shape[1:], value, device="cuda").to(t.dtype)
    full[:t.shape[0]] = t
    return full[:t.shape[0]], full


def linear(M, K, sizes):
    c = Case(M, K, sizes, [16, 32], None, seed=3, integers=True)
    c.x, _ = padded(c.x, 7.0)
    c.x8 = padded(c.x8.float(), 7.0)[1].to(torch.float8_e4m3fn)[:M]
    c.xs, _ = padded(c.xs, 7.0)
    y, full = padded(torch.zeros(M, c.N, dtype=torch.bfloat16, device="cuda"), 7.0)
    c.run(y)
    torch.cuda.synchronize()
    want = F64(y).copy()
    o = c.oracle()[0]
    small = abs(o) <= 256
    r = {"valid_err": ml.lora_read_device_error(c.ws_buf.buf),
         "valid_exact": bool((want[small] == o[small]).all())}
    if os.environ.get("MLORA_DEBUG_WAIT_FAULT"):
        return r
    # a token of segment 1 is named past the batch: it alone is lost
    c.ws_buf = ml.Workspace.for_table(c.table, M)
    pos = int(c.seg.seg_indptr[1].item()) + 2
    lost = int(c.seg.sorted_idx[pos].item())
    c.seg.sorted_idx[pos] = M + 5
    y.zero_()
    c.run(y)
    torch.cuda.synchronize()
    got = F64(y)
    keep = [m for m in range(M) if m != lost]
    r.update(err=ml.lora_read_device_error(c.ws_buf.buf),
             padding_untouched=bool((full[M:].float() == 7).all()),
             others_exact=bool((got[keep] == want[keep]).all() and (got[lost] == 0).all()))
    return r


out["decode"] = linear(40, 256, [72])
if not os.environ.get("MLORA_DEBUG_WAIT_FAULT"):
    out["groups"] = linear(150, 2048, [72])
    out["product"] = linear(150, 256, [264])
layer = Layer(M=13, E=4, topk=2, H=144, I=80, L=3, r=32)
a = layer.run()
torch.cuda.synchronize()
out["moe_err"] = ml.lora_read_device_error(layer.ws.buf)
out["moe_same"] = bool(torch.equal(a, layer.run()))
print(json.dumps(out), flush=True)
