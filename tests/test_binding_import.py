"""The binding loads, and its host-side calls run, on a torch without the e8m0 type or without a GPU build's private queries."""
import subprocess
import sys

import pytest

CODE = """
import sys
import torch
sys.path.insert(0, {root!r})
for name in {gone!r}:
    holder, _, attr = name.rpartition('.')
    obj = torch if holder == 'torch' else torch._C
    if hasattr(obj, attr):
        delattr(obj, attr)
from bit_moe_expert_top_amd import ops as L
assert L.lib.moe_mxfp8_quantize(None, 0, 32, None, None, None) == 0
assert L.moe_permute_ws_bytes(64, 8, 384) >= 0
try:
    L.moe_route_scored(torch.zeros(2, 8), 2)
except ValueError as e:
    assert 'on the GPU' in str(e)
else:
    raise SystemExit('CPU logits were taken')
print('loaded')
"""


@pytest.mark.parametrize("gone", [
    ["torch.float8_e8m0fnu"],
    ["torch.float8_e8m0fnu", "torch.float8_e4m3fn"],
    ["torch._C._cuda_getDevice", "torch._C._cuda_getCurrentRawStream"],
])
def test_import_without(gone):
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", CODE.format(root=root, gone=gone)], capture_output=True, text=True)
    assert out.returncode == 0 and "loaded" in out.stdout, out.stderr
