"""The package where torch lacks the names that the binding prefers: a torch built
without CUDA has none of them, another version may spell them otherwise."""
import subprocess
import sys

import pytest
import torch

import fp4_precision_gemms_gb300 as mx
from conftest import ROOT


def test_imports_and_refuses_on_a_torch_without_cuda():
    """The import, the size queries and the refusals need nothing of CUDA."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
torch.cuda.is_available = lambda: False
import fp4_precision_gemms_gb300 as mx
mx.build()
assert mx.norm_bwd_workspace_bytes(100, 64) > 0
x = torch.zeros(2, 32)
for call in (lambda: mx.norm_fwd(x), lambda: mx.norm_bwd(x, x, x[:, 0]), lambda: mx.act_fwd(x), lambda: mx.act_bwd(x, x),
             lambda: mx.act8_save(x), lambda: mx.act8_restore(mx.Act8.empty(2, 32, "cpu"))):
    try:
        call()
    except mx.MXError as e:
        assert e.code == mx.MX_ERR_NO_DEVICE, e
    else:
        raise AssertionError("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_public_calls_stand_in_for_the_private_ones():
    index, stream = mx._cuda_calls(object())  # none of the names
    device = torch.cuda.current_device()
    assert index() == mx._device_index() == device
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            assert stream(device) == mx._raw_stream(device) == s.cuda_stream
