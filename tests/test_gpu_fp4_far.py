"""Weights far below the largest, over the 4-bit cache: many tokens that weigh little each."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4
from paged_kv_cache_87_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,n", [(1, 131072), (1, 5000), (600, 131072), (600, 20000)])
@pytest.mark.parametrize("nats", [8.0, 16.0, 21.5, 22.5, 24.0])
@pytest.mark.parametrize("hq,d,where", [(8, 64, 0), (16, 128, 0), (4, 128, -1)])
def test_fp32_queries_count_every_token_below_a_dominant_one(hq, d, where, S, n, nats):
    """One token is `nats` above n - 1 others; its values are 0, theirs 1.  An output is then the
    others' share (n - 1) e^-nats / (1 + (n - 1) e^-nats).  A weight is held to 2^-38 of the largest
    one (absolutely) and 2^-22 relatively; logits are off by (d + 8) 2^-24 of their size, twice;
    sums of n / 64 + 100 terms by 2^-24 each; the result by 2^-24.  (One sequence is cut into many
    pieces, which weigh their tokens by themselves; of 600, each is one or two CTAs'.)"""
    B, nb = 16, 2
    k, v = (np.zeros((nb * B, 1, d), np.float32) for _ in range(2))
    k[0, 0, :] = 6.0                                       # block 0, row 0: the dominant token
    v[1:] = 6.0                                            # (6 has the code 6 and the scale 1)
    cache = [np.zeros(fp4.cache_shape(nb, 1, B, d), np.uint8) for _ in range(2)]
    for c, x in zip(cache, (k, v)):
        fp4.write(x, c, np.arange(nb * B), 1.0)
    table = torch.ones(1, -(-n // B), dtype=torch.int32)
    if where == 0:
        table[0, 0] = 0
    else:                                                  # in the last block, its first row
        table[0, (n - 1) // B] = 0
    table = table.expand(S, -1).contiguous()
    q = torch.full((S, hq, d), nats / (6 * d), dtype=torch.float32)
    got = binding.pkv_paged_decode_attention(
        q.cuda(), *(torch.from_numpy(c).cuda() for c in cache), table.cuda(),
        torch.tensor([n] * S, dtype=torch.int32, device="cuda"), n, 1.0).double().cpu() / 6
    logit = float(q[0, 0, 0].double()) * 6 * d
    w = (n - 1) * math.exp(-logit)
    want = w / (1 + w)
    rel = 2.0 ** -22 + 4 * (d + 8) * 2.0 ** -24 * nats + 2.0 ** -19 + 2 * (n / 64 + 100) * 2.0 ** -24
    tol = n * 2.0 ** -38 / (1 + w) + rel * min(want, 1 - want) * 2 + want * (n / 64 + 100) * 2.0 ** -24 + 2.0 ** -24 * want
    assert binding.pkv_get_device_status() == 0
    assert float((got - want).abs().max()) <= tol, (float(got.mean()), want, tol)
