"""First calls of a process, from several threads at once: what the library asks a device once is asked for by all."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import threading
import numpy as np
import torch
from paged_kv_cache_87_gb300 import binding
from tests.test_gpu_chunk import chunk
from tests.test_gpu_window import decode
from tests.window_cases import Paged

torch.zeros(1, device="cuda")
cases = []
for q_type, kv_type, d in (("bf16", "bf16", 128), ("f16", "e4m3", 64), ("bf16", "fp4", 128)):
    rng = np.random.default_rng(1)
    cases.append((decode, Paged(rng, [300, 5000], [1, 1], 8, 2, d, 16, q_type, kv_type, 4500, 2)))
    cases.append((chunk, Paged(rng, [300, 2000], [40, 3], 8, 2, d, 16, q_type, kv_type, 500, 2)))
    cases.append((chunk, Paged(rng, [40] * 400, [2] * 400, 8, 2, d, 16, q_type, kv_type, 30, 2)))
torch.cuda.synchronize()
got, gate = {}, threading.Barrier(4 * len(cases))

def work(i, j):
    gate.wait()
    call, c = cases[i]
    got[i, j] = call(c, stream=torch.cuda.Stream())

threads = [threading.Thread(target=work, args=(i, j)) for i in range(len(cases)) for j in range(4)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
for (i, j), out in got.items():
    cases[i][1].check(out)
    assert torch.equal(out, got[i, 0])
assert len(got) == 4 * len(cases) and binding.pkv_get_device_status() == 0
print("all right")
"""


def test_first_calls_from_many_threads():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all right" in r.stdout, r.stdout + r.stderr


CAPTURED = """
import numpy as np
import torch
from paged_kv_cache_87_gb300 import binding
from tests.test_gpu_chunk import chunk
from tests.test_gpu_window import decode
from tests.window_cases import Paged

rng = np.random.default_rng(2)
cases = [(decode, Paged(rng, [300, 5000], [1, 1], 8, 2, 128, 16, "bf16", "bf16", 4500, 2)),
         (chunk, Paged(rng, [300, 2000], [40, 3], 8, 2, 128, 16, "bf16", "e4m3", 500, 2)),
         (chunk, Paged(rng, [40] * 400, [2] * 400, 8, 2, 64, 16, "f16", "fp4", 30, 2))]
binding.load()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=side):
    outs = [call(c) for call, c in cases]
for _ in range(2):
    for out in outs:
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for (_, c), out in zip(cases, outs):
        c.check(out)
assert binding.pkv_get_device_status() == 0
print("all right")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", CAPTURED], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all right" in r.stdout, r.stdout + r.stderr
