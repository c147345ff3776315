"""The 4-bit operators called from several threads at once, and for the first time inside a capture."""
import os
import subprocess
import sys
import threading

import pytest

from gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu

FIRST_CALLS = """
import torch
from speculative_decoding_rvq_gb300 import binding as b
g = torch.Generator(device="cuda").manual_seed(5)
w = b.w4_pack(torch.randn(640, 1024, device="cuda", generator=g), 64)
x = torch.randn(24, 1024, device="cuda", generator=g).bfloat16()
y = torch.empty(24, 640, device="cuda", dtype=torch.bfloat16)
c = b.Kv4Cache(1024, 16, 2, 128)
k = torch.randn(1, 5000, 2, 128, device="cuda", generator=g)
q = torch.randn(1, 3, 8, 128, device="cuda", generator=g)
pos = torch.zeros(1, dtype=torch.int32, device="cuda")
lens = torch.full((1,), 5000, dtype=torch.int32, device="cuda")
o = torch.empty_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    b.w4_gemv(x, w, out=y)
    c.append(k, k, pos)
    c.attention(q, lens, out=o)
    held, _ = c.read(5000)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, b.w4_gemv(x, w)) and torch.equal(o, c.attention(q, lens)) and torch.equal(held, c.read(5000)[0])
assert y.any() and o.any() and held.any()
"""


def test_first_calls_inside_a_capture():
    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_several_threads_and_streams():
    """Each thread has its own stream, shapes and cache; matrix and lengths are shared.  Results are the ones a single
    thread gets."""
    require_gpu()
    from speculative_decoding_rvq_gb300 import binding as b
    g = torch.Generator(device="cuda").manual_seed(7)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    w = b.w4_pack(rand(1000, 1536), 32)
    lens = torch.tensor([3000, 77], dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")

    def work(i):
        cache = b.Kv4Cache(2 * 188, 16, 2, 64 << (i % 3))
        k, v = data[i][1:3]
        cache.append(k, v, pos)
        return [b.w4_gemv(data[i][0], w), cache.attention(data[i][3], lens), cache.read(3000)[1]]

    types = [torch.float32, torch.bfloat16, torch.float16, torch.bfloat16]
    data = [(rand(1 + 9 * i, 1536, dtype=types[i]), *(rand(2, 3000, 2, 64 << (i % 3), dtype=types[i]) for _ in range(2)),
             rand(2, 1 + 3 * i, 4, 64 << (i % 3), dtype=types[i])) for i in range(4)]
    want = [work(i) for i in range(4)]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = work(i)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001 (reported by the test's own thread)
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
