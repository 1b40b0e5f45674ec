"""Windowed decode and chunks at the ends of what scales, logits and rounding allow."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.test_gpu_chunk import chunk
from tests.test_gpu_chunk_few import many
from tests.test_gpu_window import decode
from tests.window_cases import DT, HALF, Paged

pytestmark = pytest.mark.gpu


def everywhere(rng, hq, h, d, B, q_type, kv_type, window=None, sinks=0, **kw):
    """A call of every kernel that serves these types: chunks of one and of two row tiles an item, the kernel of
    few rows, the windowed decode of one CTA a unit and of several."""
    for lens, new in (([150, 20], [90, 20]), ([300, 260], [300, 130]), many(h, [40, 21, 130], [2, 1, 3])):
        yield chunk, Paged(rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks, **kw)
    for lens in ([150, 20, 700], [30] * 400):
        yield decode, Paged(rng, lens, [1] * len(lens), hq, h, d, B, q_type, kv_type, window, sinks, **kw)


@pytest.mark.parametrize("kv_type", ["e4m3", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_zeros_under_tiny_scales_give_the_mean(kv_type, d):
    """Logits are zeros, or far below what counts, however small scale and kv_scale get."""
    rng = np.random.default_rng(d)
    cases = [("bf16", 2.0 ** -100, None), ("bf16", 2.0 ** -126, None), ("bf16", 2.0 ** -100, 2.0 ** -100),
             ("bf16", 2.0 ** -5, 2.0 ** -149), ("f16", 2.0 ** -5, 2.0 ** -149)]     # (f16 holds no smaller values)
    for q_type, kv_scale, scale in cases:
        for call, c in everywhere(rng, 4, 2, d, 16, q_type, kv_type, 60, 3, kv_scale=kv_scale):
            if scale:
                c.q = torch.from_numpy(rng.standard_normal(c.q.shape)).to(DT[q_type]).cuda()
                c.scale = scale
            c.q[2] = 0
            c.q[:, 1] = 0
            c.check(call(c))
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("kv_type", ["e4m3", "fp4"])
@pytest.mark.parametrize("kv_scale", [2.0 ** 100, 2.0 ** 60, 2.0 ** -110])
def test_bf16_rows_beside_caches_of_any_scale(kv_type, kv_scale):
    """Logits of unit spread from queries near 1 / kv_scale: rows are scaled into f16 wherever they lie."""
    rng = np.random.default_rng(1)
    for call, c in everywhere(rng, 4, 2, 128, 16, "bf16", kv_type, 60, 3, kv_scale=kv_scale):
        mul = torch.from_numpy(2.0 ** rng.integers(-12, 3, (len(c.q), 4, 1)).astype(np.float64)).cuda()
        c.q = (c.q.double() * mul).to(torch.bfloat16)
        c.check(call(c))
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("kv_type", ["f32", "e4m3", "fp4"])
@pytest.mark.parametrize("lens,window,at", [([100, 100], 50, 99), ([9000, 4000], 8000, 1500), ([3, 3], 1, 2)])
def test_a_nan_key_that_is_seen_reaches_fp32_queries(kv_type, lens, window, at):
    """... of its kv head and its sequence, and no others: alone, among pieces that are joined, and alone in sight."""
    rng = np.random.default_rng(2)
    c = Paged(rng, lens, [1] * 2, 4, 2, 128, 16, "f32", kv_type, window, 0, kv_scale=1.0 if kv_type == "f32" else 0.5)
    blk, row = int(c.table[0, at // 16]), at % 16
    if kv_type == "f32":
        c.caches[0][blk, 1, row] = float("nan")
    elif kv_type == "e4m3":
        c.caches[0].view(torch.uint8)[blk, 1, row] = 0x7F
    else:
        c.caches[0].view(-1, 2, 16 * 72)[blk, 1, 16 * 64:].view(16, 8)[row] = 0x7F     # the row's scales
    out = decode(c)
    assert torch.isnan(out[0, 2:]).all() and not torch.isnan(out[0, :2]).any()
    assert not torch.isnan(out[1]).any()
    assert binding.pkv_get_device_status() == 0


def _agreeing(q_type, kv_type, d, lens, new, hq, h, window):
    """Logits of 0 in every 16th token and x in the others, where 2^x is rounded down by nearly a whole half step of
    q_type; values of 1.  Every 16 tokens hold both, so that whoever walks them has 0 as the largest."""
    p = {"bf16": 8, "f16": 11}[q_type]
    x = np.log2(1 + 2.0 ** -p - 2.0 ** (-p - 4)) - 1           # rounds to 1/2
    c = Paged(np.random.default_rng(4), lens, new, hq, h, d, 16, q_type, kv_type, window, 0)
    for i, raw in enumerate(c.caches):
        raw = raw.view(torch.uint8) if kv_type == "e4m3" else raw
        nan = (raw[..., :1] == 0x7F) if kv_type == "e4m3" else torch.isnan(raw[..., :1])
        one = 0x38 if kv_type == "e4m3" else 1.0
        raw.zero_()
        if i == 0:
            raw[:, :, 1:, 0] = one
        else:
            raw.fill_(one)
        raw.masked_fill_(nan, 0x7F if kv_type == "e4m3" else float("nan"))
    c.q.zero_()
    c.q[:, :, 0] = -1
    c.scale = float(-x * np.log(2))
    return c


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_and_their_sum_agree(q_type, kv_type, d):
    """Rounded weights are summed as they are multiplied: the mean of equal values is that value, to the bit.  (Summed
    before they are rounded, it is off by 0.83 of a half step of the weights: 1 becomes the number below it.)"""
    for lens, window in (([160, 2000, 48], None), ([1600], 1024), ([512] * 200, 256)):
        c = _agreeing(q_type, kv_type, d, lens, [1] * len(lens), 8, 2, window)
        assert (decode(c) == 1).all(), (lens, window)
    if d == 64 or kv_type == "e4m3":
        lens, new = many(2, [160, 64, 320], [1, 1, 1])
        c = _agreeing(q_type, kv_type, d, lens, new, 8, 2, None)
        assert (chunk(c) == 1).all()
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "fp4"),
                                            ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("sign", [-1, 1])
def test_equal_logits_of_any_size_give_the_mean(q_type, kv_type, sign):
    """Keys that are all one vector: the weights are equal, whatever their logits are, up to the type's ends (chunks:
    up to 2^26, which is what the call allows)."""
    rng = np.random.default_rng(5)
    d = 64
    for log_size in (8, 20, 22, 27, 40, 120):
        # products of up to 2^log_size, 64 of them, times 1/8: from the largest queries and keys that give them
        top = {"bf16": 2.0 ** 60, "f16": 2.0 ** 15, "f32": 2.0 ** 60}[q_type]
        key = {"e4m3": 448.0, "fp4": 6.0}.get(kv_type, min(top, 2.0 ** (log_size // 2)))
        for call, c in everywhere(rng, 4, 2, d, 16, q_type, kv_type, 70, 3):
            if call is chunk and (q_type == "f32" or log_size > 22):
                continue
            raw = c.caches[0]
            if kv_type == "fp4":
                flat = raw.view(raw.shape[0], raw.shape[1], -1)
                flat[..., :16 * d // 2] = 0x77                                       # 6 and 6
                scales = flat[..., 16 * d // 2:]
                scales.masked_fill_(scales != 0x7F, 0x38)                            # 1
            elif kv_type == "e4m3":
                raw.view(torch.uint8).masked_fill_(raw.view(torch.uint8) != 0x7F, 0x7E)   # 448
            else:
                raw.masked_fill_(~torch.isnan(raw), key)
            c.q.fill_(sign * min(top, 2.0 ** log_size / key))
            out = call(c).double().cpu().numpy()
            for s, (n, m) in enumerate(zip(c.lens, c.new)):
                _, v, t = c.rows(s)
                for i in range(0, m, 7):
                    p = n - m + i
                    see = (t <= p) & ((t > p - 70) | (t < 3))
                    ref = np.repeat(v[:, see].mean(1), 2, 0)
                    step = 2.0 ** -22 if q_type == "f32" else HALF["bf16" if kv_type == "bf16" else "f16"]
                    # equal weights, rounded alike, under a sum that may be of them as they were before; sums of
                    # 73 values; one rounding
                    tol = (step + 80 * 2.0 ** -24) * np.repeat(np.abs(v[:, see]).max(1), 2, 0) + HALF[q_type] * np.abs(ref) + 1e-30
                    got = out[c.start[s] + i]
                    assert (np.abs(got - ref) <= tol).all(), (call.__name__, log_size, s, i, got[0, :3], ref[0, :3])
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("kv_type", ["e4m3", "fp4"])
def test_rows_of_one_call_from_2_to_the_minus_30_to_30(kv_type):
    """bf16 rows beside each other, each scaled by a power of two of its own; the largest have logits of unit spread."""
    rng = np.random.default_rng(6)
    for call, c in everywhere(rng, 4, 2, 128, 16, "bf16", kv_type, 60, 3, kv_scale=2.0 ** -5):
        mul = torch.from_numpy(2.0 ** rng.integers(-30, 31, (len(c.q), 4, 1)).astype(np.float64)).cuda()
        c.q = (c.q.double() * mul).to(torch.bfloat16)
        c.scale = 2.0 ** -33
        c.check(call(c))
    assert binding.pkv_get_device_status() == 0
