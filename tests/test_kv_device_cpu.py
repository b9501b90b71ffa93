"""The device that the paged cache's calls run on, with stand-ins for torch's: the
cache's device is the current one from before the stream is asked for until the
call is over, whatever the outcome, and the one before is current again."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch

seen, current = [], [3]

def exchange(i):
    seen.append(("device", i))
    was, current[0] = current[0], i
    return was

def stream(i):
    assert current[0] == i, "stream of another device than the current one"
    seen.append(("stream", i))
    if stream.fails:
        raise KeyError("no stream")
    return 0

stream.fails = False
torch._C._cuda_exchangeDevice = torch._C._cuda_maybeExchangeDevice = exchange
torch._C._cuda_getCurrentRawStream = stream
from bit_block_quantized_nibble_amd import kv

call, A, I = kv._call(), 0x10000, torch.int32
cache = bytes(kv._CCache(16, 2, 64, 16, 1, 8, A, A, None, None))
pool = bytes(kv._CPool(0, 0, 0, 17, 0, None, None, None))  # refused by its page size
K, T, L = torch.zeros(0, 2, 64, dtype=torch.bfloat16), torch.zeros(0, 8, dtype=I), torch.zeros(0, dtype=I)

def calls():  # nothing to do, or refused: none launches
    yield lambda: call.append(cache, -1, K, K, T, L, None, 0)
    yield lambda: call.attention(True, cache, -1, K, None, T, L, 0, 0, 0.1, 0, None, None, None)
    yield lambda: call.attention(False, cache, -1, K, None, T, L, 0, 0, 0.1, 0, None, None, None)
    yield lambda: call.reserve(pool, pool, -1, L, L, None, None)
    yield lambda: call.fork(cache, pool, pool, -1, L, L, None, None)
    yield lambda: call.release(pool, pool, -1, L, 0, 0)
    yield lambda: call.compact(cache, pool, pool, -1, T, None, None)

for f in calls():
    del seen[:]
    f()
    assert seen == [("device", -1), ("stream", -1), ("device", 3)] and current == [3], seen
stream.fails = True
for f in calls():
    del seen[:]
    try:
        f()
    except KeyError:
        pass
    else:
        raise AssertionError("the stream's error is lost")
    assert seen == [("device", -1), ("stream", -1), ("device", 3)] and current == [3], seen
stream.fails, current[0] = False, -1
for f in calls():  # it is the current one already
    del seen[:]
    f()
    assert seen == [("device", -1), ("stream", -1)], seen
print("fine")
"""


def test_calls_run_with_the_caches_device_current():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr
