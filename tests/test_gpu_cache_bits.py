"""Caches of the rows' own type move bits: every pattern, NaNs with their signs and payloads."""
import pytest
import torch

from paged_kv_cache_87_gb300 import binding

pytestmark = pytest.mark.gpu

KINDS = {"f16": (torch.float16, torch.int16), "bf16": (torch.bfloat16, torch.int16),
         "f32": (torch.float32, torch.int32)}


def any_bits(shape, dt, seed):
    """Random bit patterns, one in eight a NaN of either sign and any payload."""
    g = torch.Generator().manual_seed(seed)
    ints = KINDS[dt][1]
    top = {"f16": 0x7C00, "bf16": 0x7F80, "f32": 0x7F800000}[dt]
    bits = torch.iinfo(ints).bits
    x = torch.randint(0, 1 << bits, shape, generator=g)
    nan = torch.rand(shape, generator=g) < 0.125
    x = torch.where(nan, x | top | 1, x)
    x = torch.where(x >= 1 << (bits - 1), x - (1 << bits), x)
    return x.to(ints).view(KINDS[dt][0]).cuda()


@pytest.mark.parametrize("d,B,h", [(64, 8, 3), (128, 16, 2), (128, 32, 9)])
@pytest.mark.parametrize("dt", list(KINDS))
def test_every_bit_pattern_is_written_and_read_back(dt, d, B, h):
    ints = KINDS[dt][1]
    T, nb = 75, -(-75 // B) + 1
    key, value = (any_bits((T, h, d), dt, i) for i in range(2))
    assert key.isnan().any() and value.isnan().any()
    slots = torch.randperm(nb * B, generator=torch.Generator().manual_seed(2))[:T].cuda()
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    rows = torch.tensor([0, nb * B], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(nb, h, B, d, dtype=KINDS[dt][0], device="cuda") for _ in range(2))
    binding.pkv_reshape_and_cache(key, value, k, v, slots)
    out = binding.pkv_gather_cache(k, v, table, rows, nb * B, KINDS[dt][0])
    for got, x in zip(out, (key, value)):
        assert torch.equal(got[slots].view(ints), x.view(ints))
    # the fused write: values as they are, keys as the two calls give them
    cs = torch.rand(T, d, device="cuda")
    pos = torch.arange(T, device="cuda")
    k2, v2 = (torch.zeros_like(k) for _ in range(2))
    q = torch.ones_like(key)
    binding.pkv_qk_norm_rope_and_cache(q, key, value, cs, pos, k2, v2, slots)
    assert torch.equal(v2.view(ints), v.view(ints))
    turned = binding.pkv_qk_norm_rope(q, key, cs, pos)[1]
    binding.pkv_reshape_and_cache(turned, value, k, v, slots)
    assert torch.equal(k2.view(ints), k.view(ints))
    assert binding.pkv_get_device_status() == 0
