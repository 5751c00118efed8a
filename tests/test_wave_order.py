"""Lanes of a wavefront that hand each other values through LDS: the wave barrier alone
is no memory operation to the compiler, which may then move loads and stores over it.
Every such place calls stage_order(), which holds both."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adapter_lora_amd", "csrc")


def test_wave_barriers_order_memory():
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"__builtin_amdgcn_wave_barrier\(\)", text):
            found.setdefault(os.path.basename(path), []).append(text[:m.start()].rstrip())
    assert list(found) == ["row_stage.hpp"] and len(found["row_stage.hpp"]) == 1, {k: len(v) for k, v in found.items()}
    assert found["row_stage.hpp"][0].endswith('asm volatile("" ::: "memory");')
