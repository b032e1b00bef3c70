"""The first calls of a process, from eight host threads at once: each kernel's setup happens there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading, torch
import fp4_precision_gemms_gb300 as mx

T, K, F, N = 512, 512, 1024, 8
torch.manual_seed(3)
X = torch.randn(T, K, device="cuda").bfloat16()
W = (torch.randn(2 * F, K, device="cuda") / K ** 0.5).bfloat16()
dH = (torch.randn(T, F, device="cuda") * 1e-2).bfloat16()
torch.cuda.synchronize()
start = threading.Barrier(N)
got, errors = [None] * N, []

def work(i):
    try:
        fmt = ("mxfp8", "nvfp4")[i % 2]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            start.wait()
            kept = mx.gated_fwd_save(X, W, fmt)
            dX, dW = mx.gated_bwd(dH, kept, K, fmt)
            got[i] = (kept.h, dX, dW, mx.linear_fwd(X, W, fmt), mx.gated_fwd(X[:40], W, fmt))
        stream.synchronize()
    except Exception as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
for t in threads: t.start()
for t in threads: t.join()
assert not errors, errors
for i in range(2, N):
    assert all(torch.equal(a, b) for a, b in zip(got[i], got[i % 2]))
assert mx.last_device_status() == mx.MX_OK
print("same")
"""


def test_from_eight_threads():
    import fp4_precision_gemms_gb300 as mx
    mx.build()
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
