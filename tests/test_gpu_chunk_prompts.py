"""Prompts from their first token on: items of every length, dealt whole; and what stays cut beside them."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.marked_cases import Marked
from tests.test_gpu_chunk import TYPES, chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_prompts_whole_and_cut(q_type, kv_type):
    rng = np.random.default_rng(1)
    for lens, new, hq, h, d in (([1500], [1500], 8, 2, 64), ([1100, 700], [1100, 700], 16, 8, 128),
                                ([9000, 400], [300, 400], 4, 1, 128), ([6000] + [50] * 40, [30] + [50] * 40, 4, 2, 64)):
        c = Marked(rng, lens, new, hq, h, d, 16, q_type, kv_type, None, 0)
        out = chunk(c)
        assert binding.pkv_get_device_status() == 0
        c.check(out)
        assert torch.equal(out, chunk(c))


def _time(f):
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        f()
        a.record()
        for _ in range(5):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 5)
    return best


@pytest.mark.parametrize("lens", [[4096], [4000] * 4, [8192] * 2])
def test_prompts_take_what_the_multi_query_call_takes(lens):
    """The two calls that serve a 16-bit prompt of 128 dims, within a quarter."""
    B, h, hq, d = 16, 8, 32, 128
    nb = [-(-n // B) for n in lens]
    k = torch.randn(sum(nb), h, B, d, device="cuda").to(torch.bfloat16)
    table = torch.zeros(len(lens), max(nb), dtype=torch.int32)
    for s, n in enumerate(nb):
        table[s, :n] = torch.arange(sum(nb[:s]), sum(nb[:s]) + n)
    start = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
    q = torch.randn(sum(lens), hq, d, device="cuda").to(torch.bfloat16)
    args = (q, k, k, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), start, max(lens), d ** -0.5)
    assert _time(lambda: binding.pkv_paged_chunk_attention(*args)) < \
        1.25 * _time(lambda: binding.pkv_paged_multi_query_attention(*args))
    assert binding.pkv_get_device_status() == 0
