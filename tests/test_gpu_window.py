"""Decode under a sliding window with sinks, over every type of cache: against fp64, with everything
that is not seen poisoned and junk in the tables where blocks were given back."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.window_cases import DT, Paged

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3"),
         ("f32", "e4m3"), ("bf16", "fp4"), ("f16", "fp4"), ("f32", "fp4")]


def decode(c: Paged, **kw):
    return binding.pkv_paged_decode_attention_window(
        c.q, *c.caches, c.gtable, c.glens, c.most, c.scale, c.window if c.window else 2 ** 31 - 1,
        c.sinks, kv_scale=c.kv_scale, **kw)


def run(rng, lens, hq, h, d, B, q_type, kv_type, window, sinks, **kw):
    c = Paged(rng, lens, [1] * len(lens), hq, h, d, B, q_type, kv_type, window, sinks, **kw)
    out = decode(c)
    assert binding.pkv_get_device_status() == 0
    c.check(out)
    return c, out


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("d,B,window,sinks", [(128, 16, 100, 4), (64, 8, 37, 0), (128, 32, 33, 40),
                                              (64, 32, 1, 1), (128, 8, 500, 3)])
def test_types_and_windows(q_type, kv_type, d, B, window, sinks):
    rng = np.random.default_rng(d + B + window)
    lens = [1, window, window + 1, window + sinks + 1, window + B, 3 * B, 777, 1500]
    run(rng, lens, 8, 2, d, B, q_type, kv_type, window, sinks,
        kv_scale=1.0 if kv_type == q_type else 0.03125)


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("hq,h", [(1, 1), (3, 3), (10, 2), (7, 1), (16, 2), (24, 2), (40, 1), (20, 20)])
def test_head_layouts(kv_type, hq, h):
    rng = np.random.default_rng(hq * 10 + h)
    run(rng, [5, 300, 64, 1000], hq, h, 128, 16, "bf16", kv_type, 130, 2,
        kv_scale=1.0 if kv_type == "bf16" else 0.02)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
@pytest.mark.parametrize("B", [8, 16, 32])
def test_every_offset_of_the_window_in_its_blocks(q_type, kv_type, B):
    """Lengths one apart, so that the window starts at every row of a block, sinks end at every row."""
    rng = np.random.default_rng(B)
    for sinks in (0, 1, B - 1, B, B + 1):
        run(rng, list(range(3 * B, 5 * B + 2)), 2, 1, 64, B, q_type, kv_type, B + 3, sinks,
            kv_scale=1.0 if kv_type == q_type else 1.7)


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "fp4"), ("f32", "f32")])
def test_contexts_cut_into_pieces(q_type, kv_type):
    """Few long contexts: a unit is split over many CTAs; every piece of it masks its own tokens."""
    rng = np.random.default_rng(3)
    run(rng, [9000, 4000], 4, 1, 128, 16, q_type, kv_type, 8000, 20, kv_scale=1.0 if kv_type == q_type else 0.5)
    run(rng, [30011], 8, 2, 64, 32, q_type, kv_type, 4097, 5, kv_scale=1.0 if kv_type == q_type else 0.5)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_empty_contexts_give_zeros(q_type, kv_type):
    rng = np.random.default_rng(4)
    c = Paged(rng, [0, 50, 0, 3], [1] * 4, 4, 2, 64, 16, q_type, kv_type, 20, 2)
    out = torch.full_like(c.q, float("nan"))
    assert decode(c, out=out) is out and binding.pkv_get_device_status() == 0
    assert (out[0] == 0).all() and (out[2] == 0).all()
    c.check(out)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_a_window_over_everything_is_the_plain_decode(q_type, kv_type):
    """Nothing is hidden: the same bits where the plain call takes the same kernel (fp32 queries),
    else the same within what either may be off."""
    rng = np.random.default_rng(5)
    c = Paged(rng, [1, 100, 513, 2000], [1] * 4, 8, 2, 128, 16, q_type, kv_type, None, 0)
    plain = binding.pkv_paged_decode_attention(c.q, *c.caches, c.gtable, c.glens, c.most, c.scale)
    for w, s in ((2000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2000)):
        got = binding.pkv_paged_decode_attention_window(c.q, *c.caches, c.gtable, c.glens, c.most,
                                                        c.scale, w, s)
        if q_type == "f32":
            assert torch.equal(got, plain), (w, s)
        c.check(got)
    c.check(plain)
    assert binding.pkv_get_device_status() == 0


def test_lengths_and_blocks_outside_are_flagged():
    rng = np.random.default_rng(6)
    for q_type, kv_type in TYPES:
        c = Paged(rng, [400, 300], [1, 1], 4, 2, 64, 16, q_type, kv_type, 50, 2)
        lens = c.glens.clone()
        c.glens = torch.tensor([500, -3], dtype=torch.int32, device="cuda")
        out = decode(c)                                     # 400 is the most: clamped; -3: empty
        assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
        assert (out[1] == 0).all()
        c.glens = lens
        c.gtable[0, 399 // 16] = c.caches[0].shape[0]       # the window's last block
        decode(c)
        assert binding.pkv_get_device_status() == binding.DEV_BAD_BLOCK_ID


def test_infinite_and_lowest_logits():
    """Keys that give logits of the lowest values, and all-equal ones, stay finite and exact means."""
    rng = np.random.default_rng(7)
    for q_type, kv_type in (("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")):
        c = Paged(rng, [70, 300], [1, 1], 4, 2, 64, 16, q_type, kv_type, 40, 3)
        for s in range(2):
            k, v, t = c.rows(s)
            blk = torch.from_numpy(c.table[s, t // 16].astype(np.int64)).cuda()
            row = torch.from_numpy(t % 16).cuda()
            c.caches[0][blk, :, row] = 0
            c.values[0][c.table[s, t // 16], :, t % 16] = 0
        c.check(decode(c))
        big = torch.finfo(DT[q_type]).max ** 0.5 / 8
        c.q.fill_(-big)
        for s in range(2):
            k, v, t = c.rows(s)
            blk = torch.from_numpy(c.table[s, t // 16].astype(np.int64)).cuda()
            row = torch.from_numpy(t % 16).cuda()
            c.caches[0][blk, :, row] = big                  # logits of -64 big^2 / 8: all the same
        out = decode(c)
        assert torch.isfinite(out.float()).all()


def test_a_step_of_a_windowed_model_captured_and_replayed():
    """Norm, rotation and write of the new token, then the windowed decode, in one graph; lengths
    grow between replays, blocks behind the window are given back."""
    rng = np.random.default_rng(8)
    B, h, hq, d, W, S = 16, 2, 8, 128, 40, 3
    nb = 24
    k = torch.zeros(nb, h, B, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ang = torch.rand(400, d // 2, device="cuda") * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    qkv = torch.empty(1, hq + 2 * h, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = torch.full((1, 400 // B), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, binding.pkv_decode_window_workspace_bytes(1, hq, h, d, B, 400, W, S, "bf16", "bf16")),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda")

    def step():
        q, kk, vv = qkv.split([hq, h, h], 1)
        qn = binding.pkv_qk_norm_rope_and_cache(q, kk, vv, cs, pos, k, v, slot)
        binding.pkv_paged_decode_attention_window(qn, k, v, table, lens, 400, d ** -0.5, W, S,
                                                  workspace=ws, out=out)
        return qn

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            qn = step()
    torch.cuda.current_stream().wait_stream(side)
    from oracle import window as plain
    free, host = list(range(nb)), {}
    keys, values = [], []
    for n in range(1, 330):
        j = (n - 1) // B
        if j not in host:
            host[j] = free.pop(0)
        for gone in [b for b in host if (b + 1) * B <= n - W and b * B >= S]:
            free.append(host.pop(gone))
        row = np.full(400 // B, -1, np.int32)
        row[list(host)] = list(host.values())
        qkv.copy_(torch.randn(1, hq + 2 * h, d, generator=torch.Generator().manual_seed(n)))
        pos.fill_(n - 1)
        slot.fill_(host[j] * B + (n - 1) % B)
        table.copy_(torch.from_numpy(row)[None])
        lens.fill_(n)
        graph.replay()
        keys.append(k[host[j], :, (n - 1) % B].double().cpu().numpy())
        values.append(v[host[j], :, (n - 1) % B].double().cpu().numpy())
        if n % 37 == 0 or n < 4 or 40 < n < 46:
            kk, vv = np.stack(keys, 1), np.stack(values, 1)
            ref = plain.attention(qn.double().cpu().numpy(), kk, vv, d ** -0.5, W, S)
            seen = plain.seen(n, 1, W, S)[0]
            from tests.window_cases import bound
            tol = bound(qn.double().cpu().numpy(), kk[:, seen], vv[:, seen], d ** -0.5, 2.0 ** -8, ref, "bf16")
            assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all(), n
    assert binding.pkv_get_device_status() == 0 and len(free) > nb - 8


def test_another_stream_and_two_calls_at_once():
    rng = np.random.default_rng(9)
    cs = [Paged(rng, [600, 1200, 90], [1] * 3, 8, 2, 128, 16, "bf16", kv, 200, 4) for kv in ("bf16", "fp4")]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[decode(c, stream=s) for _ in range(5)] for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        for x in o:
            c.check(x)
            assert torch.equal(x, o[0])


def test_refusals():
    rng = np.random.default_rng(10)
    c = Paged(rng, [30], [1], 2, 1, 64, 16, "f16", "f16", 5, 1)
    f = lambda **kw: binding.pkv_paged_decode_attention_window(
        **{**dict(query=c.q, k_cache=c.caches[0], v_cache=c.caches[1], block_tables=c.gtable,
                  context_lens=c.glens, max_context_len=30, scale=0.1, window=5, sinks=1), **kw})
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(max_context_len=33),
               dict(scale=float("nan"))):
        with pytest.raises(binding.PagedKVError):
            f(**kw)
    for kw in (dict(window=2 ** 31), dict(query=c.q[:, :, :32]), dict(block_tables=c.gtable.long()),
               dict(v_cache=c.caches[1].to(torch.bfloat16)), dict(query=c.q.transpose(0, 1))):
        with pytest.raises(ValueError):
            f(**kw)
    c.check(f(), scale=0.1)
    wide = Paged(rng, [30], [1], 2, 1, 64, 16, "f32", "f32", 5, 1)
    with pytest.raises(binding.PagedKVError):
        decode(wide, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide.check(decode(wide))


def test_queries_of_any_magnitude():
    """bf16 queries over quantised caches are scaled into f16: heads from 2^-30 to 2^30, zeros."""
    rng = np.random.default_rng(11)
    for kv_type in ("e4m3", "fp4"):
        c = Paged(rng, [150, 90, 7], [1] * 3, 16, 2, 128, 16, "bf16", kv_type, 60, 3, kv_scale=2.0 ** -5)
        mul = torch.tensor(2.0 ** rng.integers(-30, 4, (3, 16, 1)).astype(np.float64)).cuda()
        c.q = (c.q.double() * mul).to(torch.bfloat16)
        c.q[1, 3] = 0
        c.check(decode(c))
        big = Paged(rng, [40], [1], 4, 2, 128, 16, "bf16", kv_type, 30, 0, kv_scale=2.0 ** -100)
        big.check(decode(big))
    assert binding.pkv_get_device_status() == 0


def test_nan_in_what_is_seen_is_not_hidden():
    """A NaN key or value that is seen reaches the output of its heads, and of no others."""
    rng = np.random.default_rng(12)
    for q_type, kv_type in (("bf16", "bf16"), ("f16", "e4m3"), ("f32", "f32")):
        for which in (0, 1):
            if q_type == "f32" and which == 0:
                continue                  # a sum of weights that is NaN gives zeros there, as in the plain decode
            c = Paged(rng, [100, 100], [1, 1], 4, 2, 128, 16, q_type, kv_type, 50, 2)
            blk = int(c.table[0, 99 // 16])
            raw = c.caches[which]
            if kv_type == "e4m3":
                raw.view(torch.uint8)[blk, 1, 99 % 16] = 0x7F
            else:
                raw[blk, 1, 99 % 16] = float("nan")
            out = decode(c)
            assert torch.isnan(out[0, 2:]).all() and not torch.isnan(out[0, :2]).any()
            assert not torch.isnan(out[1]).any()


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "e4m3"), ("f16", "fp4"), ("f32", "fp4")])
def test_caches_beyond_32_bits(q_type, kv_type):
    """Pools of more than 2^32 bytes each, with the blocks that are used at their end; decode and chunk."""
    from oracle import window as plain
    from tests.window_cases import bound, f64, weight_step
    h, B, d, hq, W, S = 8, 16, 128, 16, 70, 3
    row = {"bf16": 256, "e4m3": 128, "fp4": 72}[kv_type]
    nb = 2 ** 32 // (h * B * row) + 40
    rng = np.random.default_rng(13)
    small = Paged(rng, [200], [3], hq, h, d, B, q_type, kv_type, None, 0)
    # the small case's blocks, moved to the end of a large pool
    k, v = (torch.zeros((nb, *c.shape[1:]), dtype=torch.uint8 if kv_type == "fp4" else c.dtype, device="cuda")
            if kv_type != "e4m3" else torch.zeros((nb, *c.shape[1:]), dtype=torch.uint8, device="cuda").view(c.dtype)
            for c in small.caches)
    n = small.caches[0].shape[0]
    for big, c in ((k, small.caches[0]), (v, small.caches[1])):
        big.view(torch.uint8)[nb - n:] = c.view(torch.uint8)
    table = small.gtable + (nb - n)
    kk, vv, _ = small.rows(0)
    q = f64(small.q)
    ep = weight_step(q_type, kv_type)
    out = binding.pkv_paged_decode_attention_window(small.q[2:], k, v, table, small.glens, 200, small.scale, W, S)
    ref = plain.attention(q[2:], kk, vv, small.scale, W, S)
    assert (np.abs(f64(out) - ref) <= bound(q[2:], kk, vv, small.scale, ep, ref, q_type)).all()
    if q_type != "f32":
        out = binding.pkv_paged_chunk_attention(small.q, k, v, table, small.glens, small.gstart, 200, small.scale, W, S)
        ref = plain.attention(q, kk, vv, small.scale, W, S)
        assert (np.abs(f64(out) - ref) <= bound(q, kk, vv, small.scale, ep, ref, q_type)).all()
    assert binding.pkv_get_device_status() == 0
