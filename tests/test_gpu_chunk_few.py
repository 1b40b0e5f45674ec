"""The chunk attention of many sequences with few rows (up to 24 of a kv head), which a kernel of their
own takes, alone and beside longer ones: against fp64, with everything that no row sees poisoned."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.test_gpu_chunk import chunk, run
from tests.window_cases import Paged

pytestmark = pytest.mark.gpu

# what that kernel serves; other types and sizes stay with the chunk kernel
KINDS = [("bf16", "e4m3", 128), ("f16", "e4m3", 128), ("bf16", "e4m3", 64), ("f16", "e4m3", 64), ("bf16", "fp4", 128), ("f16", "fp4", 128), ("bf16", "fp4", 64),
         ("f16", "fp4", 64), ("bf16", "bf16", 64), ("f16", "f16", 64)]


def enough(h):
    """Sequences that make the five (sequence, kv head) units an SM that the kernel asks for."""
    return -(-5 * torch.cuda.get_device_properties(0).multi_processor_count // h)


def many(h, lens, new):
    """lens and new over and over, until there are enough."""
    S = max(enough(h), len(lens))
    return [lens[i % len(lens)] for i in range(S)], [new[i % len(new)] for i in range(S)]


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
@pytest.mark.parametrize("B,hq,h", [(8, 8, 2), (16, 10, 2), (8, 7, 1), (32, 72, 3), (16, 24, 24)])
def test_few_rows_of_every_layout(q_type, kv_type, d, B, hq, h):
    """Rows that fill a set of eight, that do not, and that fill three; contexts around blocks and tiles."""
    rng = np.random.default_rng(100 * hq + h + B)
    most = 24 // (hq // h)
    lens = [1, 2, 24, 63, 64, 65, 127, 128, 129, 300, 450]
    new = [min(n, int(rng.integers(1, most + 1))) for n in lens]
    run(rng, *many(h, lens, new), hq, h, d, B, q_type, kv_type)


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
@pytest.mark.parametrize("B,window,sinks", [(16, 1, 0), (32, 3, 70), (8, 63, 0), (16, 64, 65), (32, 100, 17), (8, 300, 3)])
def test_few_rows_under_a_window(q_type, kv_type, d, B, window, sinks):
    rng = np.random.default_rng(window + sinks)
    lens = [1, 5, 6, 64, 66, 71, 100, 130, 131, 132, 133, 134, 135, 136, 401, 533]
    new = [min(n, 1 + i % 6) for i, n in enumerate(lens)]
    run(rng, *many(4, lens, new), 16, 4, d, B, q_type, kv_type, window, sinks)


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(None, 0), (1000, 5)])
def test_one_unit_an_sm(q_type, kv_type, d, window, sinks):
    """As few units as the kernel takes: of 1,088 tokens, or a window of as many; fewer stay with the chunk kernel."""
    rng = np.random.default_rng(d)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for S in (-(-sms // 8), (sms - 1) // 8, -(-3 * sms // 16), 5):
        lens = rng.integers(5, 1089 if window is None else 1700, S).tolist()
        run(rng, lens, [1 + i % 5 for i in range(S)], 32, 8, d, 16, q_type, kv_type, window, sinks)


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
def test_long_contexts(q_type, kv_type, d):
    rng = np.random.default_rng(3)
    lens, new = many(24, [20, 40, 33], [5, 1, 2])
    lens[7], new[7] = 5001, 6
    lens[9], new[9] = 2999, 3
    run(rng, lens, new, 96, 24, d, 16, q_type, kv_type)
    run(rng, lens, new, 96, 24, d, 32, q_type, kv_type, 2000, 300)


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
@pytest.mark.parametrize("h,S", [(32, 30), (4, 200), (1, 1100)])
def test_few_rows_beside_longer_chunks_and_none(q_type, kv_type, d, h, S):
    """Single tokens, drafts, sequences without new tokens and one of 100: two kernels share the call, with
    every kind of planning."""
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 400 if S < 1000 else 40, S).tolist()
    new = [int(rng.integers(0, min(n, 5) + 1)) for n in lens]
    lens[S // 2], new[S // 2] = 333, 100
    lens[3], new[3] = 0, 0
    assert sum(new) * 2 <= S * 24 and S >= enough(h)
    run(rng, lens, new, 2 * h, h, d, 16, q_type, kv_type)
    run(rng, lens, new, 2 * h, h, d, 16, q_type, kv_type, 33, 5)


def test_few_rows_that_break_the_contract_are_skipped_and_flagged():
    rng = np.random.default_rng(7)
    for q_type, kv_type, d in KINDS:
        S = enough(8)
        c = Paged(rng, [60] * S, [2] * S, 16, 8, d, 16, q_type, kv_type, 50, 2)
        good, start = c.glens.clone(), c.gstart
        for n in (1, c.most + 1, -5):
            c.glens = good.clone()
            c.glens[1] = n
            out = torch.full_like(c.q, float("nan"))
            chunk(c, out=out)
            assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
            assert torch.isnan(out[2:4]).all() and not torch.isnan(out[:2]).any() and not torch.isnan(out[4:]).any()
        c.glens = good
        for at, to in ((0, -1), (0, 1), (2, 3 * S), (2, 0), (S, 2 * S - 1), (S, 2 * S + 1), (5, -2 ** 31)):
            c.gstart = start.clone()
            c.gstart[at] = to
            chunk(c)
            assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
        c.gstart = start
        c.gtable[0, 59 // 16] = c.caches[0].shape[0]
        chunk(c)
        assert binding.pkv_get_device_status() == binding.DEV_BAD_BLOCK_ID


def test_rows_behind_the_last_stay():
    rng = np.random.default_rng(6)
    lens, new = many(8, [30, 0, 50, 7], [2, 0, 0, 3])
    c = Paged(rng, lens, new, 16, 8, 64, 16, "f16", "fp4", 20, 2)
    q = torch.cat([c.q, torch.full((3, 16, 64), float("nan"), dtype=torch.float16, device="cuda")])
    out = torch.full_like(q, 5.0)
    binding.pkv_paged_chunk_attention(q, *c.caches, c.gtable, c.glens, c.gstart, c.most, c.scale, 20, 2,
                                      kv_scale=c.kv_scale, out=out)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
    assert (out[len(c.q):] == 5.0).all()
    c.check(out[:len(c.q)])


def test_nan_in_what_is_seen_is_not_hidden():
    rng = np.random.default_rng(15)
    for q_type, kv_type, d in (("bf16", "bf16", 64), ("f16", "e4m3", 128)):
        for which in (0, 1):
            lens, new = many(8, [100, 300], [3, 2])
            c = Paged(rng, lens, new, 32, 8, d, 16, q_type, kv_type, 500, 2)
            n, m = lens[0], new[0]
            blk, at = int(c.table[0, (n - m) // 16]), (n - m) % 16
            raw = c.caches[which]
            if kv_type == "e4m3":
                raw.view(torch.uint8)[blk, 1, at] = 0x7F
            else:
                raw[blk, 1, at] = float("nan")
            out = chunk(c)
            assert torch.isnan(out[:m, 4:8]).all()
            assert not torch.isnan(out[:m, :4]).any() and not torch.isnan(out[:m, 8:]).any()
            assert not torch.isnan(out[m:]).any()


def test_queries_of_any_magnitude():
    rng = np.random.default_rng(10)
    for kv_type in ("e4m3", "fp4"):
        lens, new = many(8, [150, 90], [3, 4])
        c = Paged(rng, lens, new, 32, 8, 128, 16, "bf16", kv_type, None, 0, kv_scale=2.0 ** -5)
        mul = torch.tensor(2.0 ** rng.integers(-30, 4, (len(c.q), 32, 1)).astype(np.float64)).cuda()
        c.q = (c.q.double() * mul).to(torch.bfloat16)
        c.q[3] = 0
        c.check(chunk(c))


def test_the_same_bits_every_time_captured_streamed_and_eager():
    rng = np.random.default_rng(12)
    for long in (False, True):
        lens, new = many(8, [400, 300, 200], [3, 2, 1])
        if long:
            new[1] = 70
        c = Paged(rng, lens, new, 32, 8, 128, 16, "bf16", "e4m3", None, 0, kv_scale=0.5)
        want = chunk(c)
        c.check(want)
        side = torch.cuda.Stream()
        outs = [chunk(c) for _ in range(3)] + [chunk(c, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        out = torch.empty_like(want)
        ws = torch.empty(binding.pkv_chunk_workspace_bytes(len(lens), sum(new), 32, 8, 128, c.most),
                         dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chunk(c, out=out, workspace=ws)
            chunk(c, out=out, workspace=ws)
        ws.fill_(255)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert binding.pkv_get_device_status() == 0
