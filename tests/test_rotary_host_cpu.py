"""A rotation and vectors in host memory: refused before a stream is asked for, with
nothing enqueued. Stand-ins for torch's device calls count what gets that far."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch

seen = []
torch._C._cuda_exchangeDevice = torch._C._cuda_maybeExchangeDevice = lambda i: seen.append(i) or -1
torch._C._cuda_getCurrentRawStream = lambda i: seen.append(i) or 0
import bit_block_quantized_nibble_amd as qbn
from bit_block_quantized_nibble_amd import kv

kv._call()
r = qbn.Rope([1.0] * 8, device="cpu")
for dt in (torch.float32, torch.bfloat16):
    for tokens, heads, dim in ((0, 1, 16), (0, 0, 32), (3, 0, 8), (3, 2, 24), (3, 2, 8)):  # none of them reaches a launch
        x = torch.ones(tokens, heads, dim, dtype=dt)
        for out in (None, x):
            try:
                qbn.rope(x, torch.zeros(tokens, dtype=torch.int32), r, out=out)
            except ValueError as e:
                assert "must be on a device (cuda)" in str(e) and "cpu" in str(e), e
            else:
                raise AssertionError("host tensors were taken")
assert not seen, seen
print("fine")
"""


def test_host_tensors_are_refused():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr
