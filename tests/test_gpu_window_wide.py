"""Decodes under windows of many tokens and few units: no slower than the plain decode of as many."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.marked_cases import Marked
from tests.test_gpu_window import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "e4m3"), ("f16", "fp4"), ("f32", "f32")])
@pytest.mark.parametrize("hq,h,d", [(4, 1, 128), (24, 2, 64)])
def test_every_number_of_tiles_and_sequences_around_the_widest_clusters(q_type, kv_type, hq, h, d):
    rng = np.random.default_rng(hq)
    for lens, window in (([4032], None), ([4033, 1], 2 ** 31 - 1), ([4097, 64, 0, 1025], 4096), ([9001, 30, 5000], 8500),
                         ([5000] * 9, 4500), ([4200] * 20, 4200)):
        c = Marked(rng, lens, [1] * len(lens), hq, h, d, 16, q_type, kv_type, window if window and window < 2 ** 31 - 1 else None, 0)
        out = decode(c)
        assert binding.pkv_get_device_status() == 0
        assert all((out[s] == 0).all() for s, n in enumerate(lens) if n == 0)
        keep = [s for s, n in enumerate(lens) if n]
        c.lens, c.new, c.start = [lens[s] for s in keep], [1] * len(keep), np.arange(len(keep) + 1)
        c.check(out[keep])


def _time(f):
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        f()
        a.record()
        for _ in range(10):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 10)
    return best


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,h", [(8, 1), (64, 8)])
def test_one_sequence_of_many_tokens(kv_type, hq, h):
    """A window over all of 131,072 tokens costs no more than the plain decode (a tenth for the clock)."""
    n, B, d = 131072, 16, 128
    dt = torch.bfloat16 if kv_type == "bf16" else torch.float8_e4m3fn
    k = torch.ones(n // B, h, B, d, device="cuda").to(dt)
    v = k.clone()
    q = torch.ones(1, hq, d, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(n // B, device="cuda").to(torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    args = (q, k, v, table, lens, n, d ** -0.5)
    windowed = _time(lambda: binding.pkv_paged_decode_attention_window(*args, 2 ** 31 - 1))
    assert windowed < 1.1 * _time(lambda: binding.pkv_paged_decode_attention(*args))
    assert (binding.pkv_paged_decode_attention_window(*args, 2 ** 31 - 1) == 1).all()
    assert binding.pkv_get_device_status() == 0
