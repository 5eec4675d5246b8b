"""hc_device_error costs a process that makes no call of the attention sublayer what it did without them: the words of kernels
that were never launched are not fetched."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PROGRAM = """
import time
import torch
import hyper_connection_residual_hc_gb300 as hc

torch.zeros(1, device="cuda")

def cost():
    times = []
    for _ in range(300):
        t = time.perf_counter()
        assert hc.hc_device_error(clear=True) == 0
        times.append(time.perf_counter() - t)
    return sorted(times)[len(times) // 2]

without = cost()
shape = hc.kv_shape(4, 64, 1, 64)
cache = torch.zeros(hc.hc_kv_cache_size(shape), dtype=torch.uint8, device="cuda")
x = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
slots = torch.arange(64, device="cuda")
hc.hc_kv_write(x, 64, x, 64, slots, 64, shape, cache)
ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
out, ws = torch.empty_like(x), hc.new_kv_workspace()
for n in (1, 64):  # by either kernel
    hc.hc_kv_attention(x, 64, ints(0, n), ints(64), ints(0), cache, hc.attention(n, 1, n, 1, 1, 1.0), shape, out, 64, None, ws)
beside = cost()
hc.hc_kv_write(x, 64, x, 64, slots + 10 ** 6, 64, shape, cache)
assert hc.hc_device_error(clear=True) == 1 << 20
for n in (1, 64):
    hc.hc_kv_attention(x, 64, ints(0, n), ints(65), ints(0), cache, hc.attention(n, 1, n, 1, 1, 1.0), shape, out, 64, None, ws)
    assert hc.hc_device_error(clear=True) == 1 << 21
print("without %.1f us, beside %.1f us" % (1e6 * without, 1e6 * beside))
assert without < 0.75 * beside  # 2 words of 5
"""


def test_words_of_kernels_never_launched_are_not_fetched():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
