"""Attention of chunks of new tokens over caches of 16 bits, FP8 and 4 bits, causal or under a window
with sinks: against fp64, with everything that no row sees poisoned."""
import numpy as np
import pytest
import torch

from oracle import window as plain
from paged_kv_cache_87_gb300 import binding
from tests.window_cases import Paged, bound, f64, weight_step

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "fp4"), ("f16", "fp4")]


def chunk(c: Paged, **kw):
    return binding.pkv_paged_chunk_attention(c.q, *c.caches, c.gtable, c.glens, c.gstart, c.most, c.scale,
                                             c.window, c.sinks, kv_scale=c.kv_scale, **kw)


def run(rng, lens, new, hq, h, d, B, q_type, kv_type, window=None, sinks=0, **kw):
    kw.setdefault("kv_scale", 1.0 if kv_type == q_type else 0.03125)
    c = Paged(rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks, **kw)
    out = chunk(c)
    assert binding.pkv_get_device_status() == 0
    c.check(out)
    return c, out


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_one_tile(q_type, kv_type, d):
    rng = np.random.default_rng(d)
    run(rng, [5], [5], 1, 1, d, 16, q_type, kv_type)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("d,B", [(64, 8), (128, 16), (128, 32), (64, 32), (128, 8)])
def test_causal_chunks(q_type, kv_type, d, B):
    rng = np.random.default_rng(d + B)
    run(rng, [1, 129, 200, 40, 700, 1000], [1, 129, 33, 40, 5, 300], 8, 2, d, B, q_type, kv_type)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("d,B,window,sinks", [(128, 16, 100, 4), (64, 8, 37, 0), (128, 32, 1, 1),
                                              (64, 16, 300, 140), (128, 8, 129, 5)])
def test_chunks_under_a_window(q_type, kv_type, d, B, window, sinks):
    rng = np.random.default_rng(window)
    run(rng, [1, 129, 200, 40, 700, 1000, 1600], [1, 129, 33, 40, 5, 300, 1], 8, 2, d, B, q_type, kv_type,
        window, sinks)


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("hq,h", [(1, 1), (3, 3), (10, 2), (7, 1), (48, 2), (128, 1), (66, 1), (20, 20)])
def test_head_layouts(kv_type, hq, h):
    """Groups that divide 128 and that do not, up to a row tile a token."""
    rng = np.random.default_rng(hq * 10 + h)
    run(rng, [9, 260, 300], [9, 37, 3], hq, h, 128, 16, "bf16", kv_type, 130, 2)
    run(rng, [70, 150], [70, 2], hq, h, 64, 8, "bf16", kv_type)


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "fp4")])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_every_offset_in_blocks_and_tiles(q_type, kv_type, B):
    """Lengths, chunks and windows around blocks and tiles of 128."""
    rng = np.random.default_rng(B)
    for window, sinks in ((B + 3, 1), (127, B), (128, B + 1), (129, 129), (256, 127)):
        lens = [120 + 7 * i for i in range(12)] + [254, 255, 256, 257, 384, 385]
        new = [1 + 11 * i % 64 for i in range(len(lens))]
        run(rng, lens, new, 2, 1, 64, B, q_type, kv_type, window, sinks)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_items_cut_over_many_sms(q_type, kv_type):
    """Few rows over long contexts: every item lies in many runs, and is joined."""
    rng = np.random.default_rng(3)
    run(rng, [20011], [3], 4, 1, 128, 16, q_type, kv_type)
    run(rng, [9000, 7000, 100], [70, 1, 100], 8, 2, 64, 32, q_type, kv_type)
    run(rng, [9000, 7000], [70, 300], 4, 1, 128, 8, q_type, kv_type, 5000, 300)


@pytest.mark.parametrize("kv_type", ["bf16", "fp4"])
def test_whole_items_from_the_counter(kv_type):
    """Many short items: more than the SMs, so none is cut."""
    rng = np.random.default_rng(4)
    S = 300
    lens = rng.integers(1, 90, S).tolist()
    new = [int(rng.integers(1, n + 1)) for n in lens]
    run(rng, lens, new, 8, 4, 64, 16, "bf16", kv_type, 40, 2)


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "fp4")])
@pytest.mark.parametrize("window,sinks", [(None, 0), (150, 3)])
def test_whole_items_of_two_tiles_from_the_counter(q_type, kv_type, window, sinks):
    rng = np.random.default_rng(40)
    S = 30
    lens = rng.integers(100, 600, S).tolist()
    new = [int(rng.integers(60, min(n, 200))) for n in lens]
    run(rng, lens, new, 16, 4, 64, 16, q_type, kv_type, window, sinks)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 9])
def test_few_rows_of_every_number_of_steps(q_type, kv_type, steps):
    """Items of one row tile, whose steps the two halves of a CTA take in turn."""
    rng = np.random.default_rng(steps)
    S = 170                                            # more items than CTAs: none is cut
    run(rng, [128 * steps - int(rng.integers(0, 100)) for _ in range(S)], [2] * S, 2, 1, 64, 16, q_type, kv_type)


def test_many_sequences():
    """More sequences than the planner ranks, empty ones among them."""
    rng = np.random.default_rng(5)
    S = 1500
    lens = rng.integers(0, 20, S).tolist()
    new = [int(rng.integers(0, n + 1)) for n in lens]
    run(rng, lens, new, 2, 1, 64, 8, "bf16", "e4m3", 7, 1)


def test_sequences_without_new_tokens_and_rows_behind_the_last():
    rng = np.random.default_rng(6)
    c = Paged(rng, [30, 0, 50, 7], [3, 0, 0, 7], 4, 2, 64, 16, "f16", "fp4", 20, 2)
    q = torch.cat([c.q, torch.full((3, 4, 64), float("nan"), dtype=torch.float16, device="cuda")])
    out = torch.full_like(q, 5.0)
    # three rows behind the last sequence: total_q is flagged as another than query_start says
    binding.pkv_paged_chunk_attention(q, *c.caches, c.gtable, c.glens, c.gstart, c.most, c.scale, 20, 2,
                                      kv_scale=c.kv_scale, out=out)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
    assert (out[10:] == 5.0).all()
    c.check(out[:10])
    none = Paged(rng, [5], [0], 4, 2, 64, 16, "f16", "fp4", 20, 2)
    assert chunk(none).shape == (0, 4, 64) and binding.pkv_get_device_status() == 0


def test_sequences_that_break_the_contract_are_skipped_and_flagged():
    rng = np.random.default_rng(7)
    for q_type, kv_type in TYPES:
        c = Paged(rng, [40, 60, 80], [10, 20, 30], 4, 2, 64, 16, q_type, kv_type, 50, 2)
        good = c.glens.clone()
        for lens in ([40, 19, 80], [40, 81, 80], [40, -5, 80]):
            c.glens = torch.tensor(lens, dtype=torch.int32, device="cuda")
            out = torch.full_like(c.q, float("nan"))
            chunk(c, out=out)
            assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
            assert torch.isnan(out[10:30]).all() and not torch.isnan(out[:10]).any()
        c.glens = good
        # starts that run back and forth list rows many times over: nothing is done then, or the
        # sequences that still make sense
        start = c.gstart
        for bad in ([0, 60, 0, 60], [0, 61, 60, 60], [-1, 10, 30, 60]):
            c.gstart = torch.tensor(bad, dtype=torch.int32, device="cuda")
            chunk(c)
            assert binding.pkv_get_device_status() & binding.DEV_BAD_CONTEXT
        c.gstart = start
        c.gtable[0, 39 // 16] = c.caches[0].shape[0]
        chunk(c)
        assert binding.pkv_get_device_status() == binding.DEV_BAD_BLOCK_ID


def test_many_overlapping_starts_stay_inside_the_workspace():
    """Starts that go back and forth over 700 sequences would list 350 x 600 rows."""
    rng = np.random.default_rng(8)
    S, T = 700, 600
    q = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(40, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(S, 40, dtype=torch.int32, device="cuda")
    lens = torch.full((S,), 600, dtype=torch.int32, device="cuda")
    start = torch.tensor([0 if i % 2 == 0 else T for i in range(S + 1)], dtype=torch.int32, device="cuda")
    need = binding.pkv_chunk_workspace_bytes(S, T, 2, 1, 64, 600)
    ws = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    ws[need:] = 77
    binding.pkv_paged_chunk_attention(q, k, k, table, lens, start, 600, 0.1, workspace=ws[:need])
    assert binding.pkv_get_device_status() & binding.DEV_BAD_CONTEXT
    assert (ws[need:] == 77).all()


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_single_tokens_agree_with_the_decode(q_type, kv_type):
    rng = np.random.default_rng(9)
    c = Paged(rng, [1, 300, 77, 2000], [1] * 4, 16, 2, 128, 16, q_type, kv_type, 256, 4, kv_scale=0.25 if
              kv_type in ("e4m3", "fp4") else 1.0)
    a = chunk(c)
    b = binding.pkv_paged_decode_attention_window(c.q, *c.caches, c.gtable, c.glens, c.most, c.scale, 256, 4,
                                                  kv_scale=c.kv_scale)
    c.check(a)
    c.check(b)
    assert binding.pkv_get_device_status() == 0


def test_queries_of_any_magnitude():
    """bf16 queries over quantised caches are scaled into f16: rows from 2^-30 to 2^30, zeros."""
    rng = np.random.default_rng(10)
    for kv_type in ("e4m3", "fp4"):
        c = Paged(rng, [150], [90], 4, 2, 128, 16, "bf16", kv_type, None, 0, kv_scale=2.0 ** -5)
        mul = torch.tensor(2.0 ** rng.integers(-30, 4, (90, 4, 1)).astype(np.float64)).cuda()
        c.q = (c.q.double() * mul).to(torch.bfloat16)
        c.q[3] = 0
        c.check(chunk(c))
        big = Paged(rng, [40], [40], 4, 2, 128, 16, "bf16", kv_type, None, 0, kv_scale=2.0 ** -100)
        big.q.mul_(1.0)
        out = chunk(big)
        big.check(out)


def test_nan_in_what_is_seen_is_not_hidden():
    rng = np.random.default_rng(15)
    for q_type, kv_type in (("bf16", "bf16"), ("f16", "e4m3")):
        for which in (0, 1):
            for lens, new in (([100, 300], [60, 2]), ([3000], [40]), ([4000], [2])):
                c = Paged(rng, lens, new, 4, 2, 128, 16, q_type, kv_type, 500, 2)
                n, m = lens[0], new[0]
                blk, at = int(c.table[0, (n - m) // 16]), (n - m) % 16
                raw = c.caches[which]
                if kv_type == "e4m3":
                    raw.view(torch.uint8)[blk, 1, at] = 0x7F
                else:
                    raw[blk, 1, at] = float("nan")
                out = chunk(c)
                assert torch.isnan(out[:m, 2:]).all() and not torch.isnan(out[:m, :2]).any()
                assert not torch.isnan(out[m:]).any()


def test_outputs_that_are_16_byte_aligned():
    rng = np.random.default_rng(11)
    c = Paged(rng, [140], [140], 2, 1, 64, 16, "bf16", "bf16", None, 0)
    room = torch.zeros(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view(c.q.shape)
    chunk(c, out=out)
    c.check(out)


def test_the_same_bits_every_time_captured_streamed_and_eager():
    rng = np.random.default_rng(12)
    c = Paged(rng, [4000, 300, 2000], [40, 300, 1], 8, 2, 128, 16, "bf16", "e4m3", None, 0, kv_scale=0.5)
    want = chunk(c)
    c.check(want)
    side = torch.cuda.Stream()
    outs = [chunk(c) for _ in range(3)] + [chunk(c, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(want)
    ws = torch.empty(binding.pkv_chunk_workspace_bytes(3, 341, 8, 2, 128, c.most), dtype=torch.uint8, device="cuda")
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


def test_a_prompt_in_chunks_then_steps_over_a_4_bit_cache():
    """As a model with windowed layers uses them: write a chunk, attend, and so on, then single tokens."""
    rng = np.random.default_rng(13)
    B, h, hq, d, W, S, kv = 16, 2, 8, 128, 90, 4, 0.125
    n, nb = 400, 30
    x = torch.from_numpy(rng.standard_normal((n, hq + 2 * h, d))).to(torch.bfloat16).cuda()
    q, k, v = (t.contiguous() for t in x.split([hq, h, h], 1))
    kc, vc = (torch.full(binding.fp4_cache_shape(nb, h, B, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    m = binding.BlockManager(nb, B)
    m.add_sequence(0, n)
    table, _ = m.sequence(0)
    gt = torch.tensor([table], dtype=torch.int32, device="cuda")
    slots = torch.tensor([table[t // B] * B + t % B for t in range(n)], device="cuda")
    outs = []
    at = 0
    for size in (150, 1, 129, 60, 1, 1, 58):
        end = at + size
        binding.pkv_reshape_and_cache(k[at:end], v[at:end], kc, vc, slots[at:end], kv_scale=kv)
        lens = torch.tensor([end], dtype=torch.int32, device="cuda")
        if size == 1:
            o = binding.pkv_paged_decode_attention_window(q[at:end], kc, vc, gt, lens, n, d ** -0.5, W, S, kv_scale=kv)
        else:
            o = binding.pkv_paged_chunk_attention(q[at:end], kc, vc, gt, lens,
                                                  torch.tensor([0, size], dtype=torch.int32, device="cuda"), n,
                                                  d ** -0.5, W, S, kv_scale=kv)
        outs.append(o)
        at = end
    assert at == n and binding.pkv_get_device_status() == 0
    keys, values = binding.pkv_gather_cache(kc, vc, gt, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n,
                                            torch.float32, kv)
    kk, vv = (f64(t).transpose(1, 0, 2) for t in (keys, values))
    ref = plain.attention(f64(q), kk, vv, d ** -0.5, W, S)
    tol = bound(f64(q), kk, vv, d ** -0.5, weight_step("bf16", "fp4"), ref, "bf16")
    assert (np.abs(f64(torch.cat(outs)) - ref) <= tol).all()


def test_refusals():
    rng = np.random.default_rng(14)
    c = Paged(rng, [30, 40], [5, 6], 2, 1, 64, 16, "f16", "f16", 5, 1)
    args = dict(query=c.q, k_cache=c.caches[0], v_cache=c.caches[1], block_tables=c.gtable, context_lens=c.glens,
                query_start=c.gstart, max_context_len=40, scale=0.1, window=5, sinks=1)
    f = lambda **kw: binding.pkv_paged_chunk_attention(**{**args, **kw})
    for kw in (dict(window=0), dict(sinks=-1), dict(max_context_len=49), dict(scale=0.0), dict(scale=-1.0),
               dict(query=c.q.float()), dict(query=c.q.to(torch.bfloat16)),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(binding.PagedKVError):
            f(**kw)
    for kw in (dict(window=2 ** 31), dict(query=c.q[:, :, :32]), dict(block_tables=c.gtable.long()),
               dict(v_cache=c.caches[1].to(torch.bfloat16)), dict(query=c.q.transpose(0, 1)),
               dict(query_start=c.gstart[:2]), dict(out=c.q[:5]), dict(block_tables=c.gtable[:1])):
        with pytest.raises(ValueError):
            f(**kw)
    c.check(f(), scale=0.1)
