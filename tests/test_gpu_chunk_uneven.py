"""Many sequences of few rows and few that are much longer: the long ones leave the kernel of few rows, which does
not cut contexts, for the one that does."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.marked_cases import Marked
from tests.test_gpu_chunk import chunk
from tests.test_gpu_chunk_few import KINDS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
@pytest.mark.parametrize("h,S", [(26, 31), (8, 110), (1, 1100)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (6000, 20)])
def test_long_contexts_among_many_short_ones(q_type, kv_type, d, h, S, window, sinks):
    """Around the length that decides, at it and far beyond, with every kind of planning; a chunk of 40 rows beside."""
    rng = np.random.default_rng(S)
    lens = rng.integers(20, 60, S).tolist()
    new = rng.integers(0, 6, S).tolist()
    for s, n in ((3, 2048), (S // 2, 2100), (5, 2500), (9, 5000), (S - 1, 20011 if h < 8 else 7003)):
        lens[s], new[s] = n, 1 + s % 5
    lens[7], new[7] = 60, 40
    c = Marked(rng, lens, new, 4 * h, h, d, 16, q_type, kv_type, window, sinks)
    out = chunk(c)
    assert binding.pkv_get_device_status() == 0
    c.check(out)
    assert torch.equal(out, chunk(c))


def _time(lens, kv_type, d):
    h, B = 8, 16
    nb = sum(-(-n // B) for n in lens)
    if kv_type == "fp4":
        k = torch.full((nb, h, B, 9 * d // 16), 0x30, dtype=torch.uint8, device="cuda")
    else:
        k = torch.ones(nb, h, B, d, device="cuda").to(torch.float8_e4m3fn if kv_type == "e4m3" else torch.bfloat16)
    table = torch.zeros(len(lens), -(-max(lens) // B), dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // B)
        table[s, :m] = torch.arange(at, at + m)
        at += m
    q = torch.ones(5 * len(lens), 32, d, dtype=torch.bfloat16, device="cuda")
    args = (q, k, k, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.arange(0, 5 * len(lens) + 1, 5, dtype=torch.int32, device="cuda"), max(lens), 0.1)
    best = float("inf")
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        binding.pkv_paged_chunk_attention(*args)
        a.record()
        for _ in range(4):
            binding.pkv_paged_chunk_attention(*args)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 4)
    return best


@pytest.mark.parametrize("kv_type,d", [("e4m3", 128), ("fp4", 128), ("bf16", 64)])
def test_one_long_context_does_not_hold_up_the_others(kv_type, d):
    """A call of both takes no more than twice what the two take one after the other."""
    short = [50 + 37 * i % 350 for i in range(200)]
    assert _time(short + [131072], kv_type, d) < 2 * (_time(short, kv_type, d) + _time([131072], kv_type, d))
    assert binding.pkv_get_device_status() == 0
