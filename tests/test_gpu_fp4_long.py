"""Decode over the 4-bit cache where a CTA plans many tiles and contexts are cut into many
pieces: tables draw their blocks from a small pool, references are fp64 on the GPU."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4
from paged_kv_cache_87_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a step of rounding, relative to the value
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def pool_of(rng, nb, h, B, d):
    """A cache of quantised normal rows on the GPU, and its values in fp64."""
    c = np.zeros(fp4.cache_shape(nb, h, B, d), np.uint8)
    fp4.write((rng.standard_normal((nb * B, h, d)) * 32).astype(np.float32), c, np.arange(nb * B), 1.0)
    return torch.from_numpy(c).cuda(), torch.from_numpy(fp4.values(c, d, 1.0)).cuda()


def rows_of(vals, table, n):
    """[h, n, d] rows of a sequence's first n tokens from pool values [nb, h, B, d]."""
    h, B, d = vals.shape[1:]
    x = vals[table[:-(-n // B)].long()]                    # [blocks, h, B, d]
    return x.transpose(0, 1).reshape(h, -1, d)[:, :n]


def check(got, q, kv, vv, table, lens, scale, dt):
    """Every output against fp64.  Weights have half a step of 2^-11 (2^-22 in two terms, for fp32
    queries) in numerator and denominator; logits are fp32 sums of d terms, off by (d + 8) 2^-24
    of the largest sum |q k| scale, which moves a weight (against the maximum) by twice that, its
    exponential 2^-21 more; a worker sums 16 tokens at a time in each of four warps and its own and
    up to 65 others' states are joined: (n / 64 + 100) 2^-24 of sum p |v|, twice; weights far below
    the largest are off by 2^-32 of it; one rounding of the result."""
    h = kv.shape[1]
    for s, n in enumerate(lens):
        if n == 0:
            assert (got[s] == 0).all()
            continue
        k, v = rows_of(kv, table[s], n), rows_of(vv, table[s], n)
        x = q[s].double().view(h, -1, q.shape[2])
        z = torch.einsum("hgd,hnd->hgn", x, k) * scale
        p = torch.softmax(z, -1)
        ref = torch.einsum("hgn,hnd->hgd", p, v)
        size = torch.einsum("hgn,hnd->hgd", p, v.abs())
        logit = (torch.einsum("hgd,hnd->hgn", x.abs(), k.abs()).amax(-1) * abs(scale))[..., None]
        rel = 2 * (2.0 ** -22 if dt == "f32" else 2.0 ** -11) + 4 * (q.shape[2] + 8) * 2.0 ** -24 * logit + \
            2.0 ** -19 + 2 * (n / 64 + 100) * 2.0 ** -24
        far = 2.0 ** -32 * v.abs().sum(1)[:, None]
        tol = (rel * size + far) * (1 + HALF[dt]) + HALF[dt] * ref.abs() + 1e-30
        err = (got[s].double().view_as(ref) - ref).abs()
        assert (err <= tol).all(), (s, n, float((err / tol).max()))


@pytest.mark.parametrize("hq,h,d,B,dt", [(16, 8, 64, 16, "bf16"), (16, 8, 128, 8, "f16"), (40, 4, 64, 32, "f32")])
def test_decode_plans_of_several_rounds_repeat_their_bits(hq, h, d, B, dt):
    """More units than a CTA plans at once (32 slots, one a lane), three rounds and more each."""
    rng = np.random.default_rng(hq + d)
    S, nb = 3000, 64
    lens = rng.integers(0, 260, S)
    table = torch.from_numpy(rng.integers(0, nb, (S, -(-260 // B))).astype(np.int32)).cuda()
    (gk, kv), (gv, vv) = (pool_of(rng, nb, h, B, d) for _ in range(2))
    q = (torch.from_numpy(rng.standard_normal((S, hq, d))) / 32).to(DT[dt]).cuda()
    args = (q, gk, gv, table, torch.from_numpy(lens.astype(np.int32)).cuda(), 260, 1 / math.sqrt(d))
    out = binding.pkv_paged_decode_attention(*args)
    check(out, q, kv, vv, table, lens.tolist(), 1 / math.sqrt(d), dt)
    for _ in range(20):
        assert torch.equal(out, binding.pkv_paged_decode_attention(*args))
    assert binding.pkv_get_device_status() == 0


LONG = [  # hq, h, d, B, dt, lens: one context in some 60 pieces (joined by sixteen warps), units of
          # sixteen heads, and more units than a CTA each, cut where runs end (joined by eight warps)
    (8, 1, 64, 32, "bf16", [100000]), (4, 1, 128, 16, "f32", [100000, 0, 3]),
    (16, 1, 128, 16, "f16", [20000, 0, 9000, 1, 40]), (12, 1, 64, 8, "f32", [9000, 20000]),
    (20, 1, 128, 32, "bf16", [70000]), (16, 8, 64, 16, "bf16", "many"), (64, 4, 128, 16, "f16", "many"),
    (24, 8, 128, 8, "f32", "many")]


def lens_of(lens, rng):
    if lens != "many":
        return lens
    x = np.exp(rng.uniform(0, math.log(9500), 60)).astype(int)
    x[3], x[17], x[40] = 9500, 0, 8193
    return x.tolist()


@pytest.mark.parametrize("hq,h,d,B,dt,lens", LONG)
def test_decode_joins_contexts_cut_into_many_pieces(hq, h, d, B, dt, lens):
    """Equal runs and the joining kernel, eagerly and replayed over a workspace of any contents."""
    rng = np.random.default_rng(hq + h + d)
    lens = lens_of(lens, rng)
    S, nb, most = len(lens), 97, max(lens)
    assert most > 8192                                     # (bounds up to that may take clusters)
    table = torch.from_numpy(rng.integers(0, nb, (S, -(-most // B))).astype(np.int32)).cuda()
    (gk, kv), (gv, vv) = (pool_of(rng, nb, h, B, d) for _ in range(2))
    q = (torch.from_numpy(rng.standard_normal((S, hq, d))) / 32).to(DT[dt]).cuda()
    args = (q, gk, gv, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), most, 1 / math.sqrt(d))
    out = binding.pkv_paged_decode_attention(*args)
    check(out, q, kv, vv, table, lens, 1 / math.sqrt(d), dt)
    ws = torch.empty(binding.pkv_decode_workspace_bytes(S, hq, h, d, B, most, "e2m1"), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(out)
    binding.pkv_paged_decode_attention(*args, workspace=ws, out=got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.pkv_paged_decode_attention(*args, workspace=ws, out=got)
    for fill in (0, 255, 127):
        ws.fill_(fill), got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    assert torch.equal(binding.pkv_paged_decode_attention_noalloc(*args), out)
    # other lengths in the same buffers, replayed: other cuts
    other = lens[1:] + [most // 2]
    args[4].copy_(torch.tensor(other, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(got, q, kv, vv, table, other, 1 / math.sqrt(d), dt)
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("hq,h,d,B,dt,lens", LONG + [(8, 2, 128, 16, "bf16", [8000, 0, 700, 129])])
def test_decode_counts_every_tile_once(hq, h, d, B, dt, lens):
    """A scale of 0 weighs every token alike, and a tile's values are 6 in one dim: an output is 6
    times the share of the tokens marked so.  Weights are one power of two and sums whole multiples
    of it below 2^24: exact; the quotient and the product round by 2^-24 each, then the result."""
    rng = np.random.default_rng(hq + d)
    lens = lens_of(lens, rng)
    S, most = len(lens), max(lens)
    gk, _ = pool_of(rng, d, h, B, d)
    x = np.zeros((d, B, h, d), np.float32)
    x[np.arange(d), :, :, np.arange(d)] = 6.0              # block j: dim j
    c = np.zeros(fp4.cache_shape(d, h, B, d), np.uint8)
    fp4.write(x.reshape(d * B, h, d), c, np.arange(d * B), 1.0)
    marks = rng.integers(0, d, (S, -(-most // 128)))
    table = np.repeat(marks, 128 // B, 1)[:, :-(-most // B)].astype(np.int32)
    q = torch.randn(S, hq, d, device="cuda").to(DT[dt])
    out = binding.pkv_paged_decode_attention(
        q, gk, torch.from_numpy(c).cuda(), torch.from_numpy(np.ascontiguousarray(table)).cuda(),
        torch.tensor(lens, dtype=torch.int32, device="cuda"), most, 0.0).double().cpu().numpy()
    assert binding.pkv_get_device_status() == 0
    for s, n in enumerate(lens):
        tiles = -(-n // 128)
        tokens = np.minimum(128, n - 128 * np.arange(tiles))
        want = 6.0 * np.bincount(marks[s, :tiles], weights=tokens, minlength=d) / max(n, 1)
        tol = want * (HALF[dt] + 2.0 ** -22)
        if dt == "f16":
            tol = tol + 2.0 ** -25                         # half a step of its smallest values
        assert (np.abs(out[s] - want) <= tol).all(), (s, n)


def test_decode_of_a_context_of_all_31_bits():
    """2^31 - 1 tokens, and 127 fewer, over a table that repeats 64 blocks marked with a dim each.
    Every weight is alike; a warp's sums are whole and below 2^24, and some 70 of them are added:
    128 2^-24 at most; 127 tokens more or less are 2^-18 of an output; then the result's rounding."""
    n, d, B = (1 << 31) - 1, 64, 32
    x = np.zeros((d, B, 1, d), np.float32)
    x[np.arange(d), :, :, np.arange(d)] = 6.0
    c = np.zeros(fp4.cache_shape(d, 1, B, d), np.uint8)
    fp4.write(x.reshape(d * B, 1, d), c, np.arange(d * B), 1.0)
    cache = torch.from_numpy(c).cuda()
    g = torch.Generator("cuda").manual_seed(4)
    table = torch.randint(0, d, (1, 1 << 26), generator=g, dtype=torch.int32, device="cuda")
    want = 6.0 * B * torch.bincount(table[0], minlength=d).double()
    want[table[0, -1]] -= 6.0
    want /= n
    q = torch.randn(1, 8, d, device="cuda").bfloat16()
    for length in (n, n - 127):
        out = binding.pkv_paged_decode_attention(q, cache, cache, table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                                                 n, 0.0)
        assert binding.pkv_get_device_status() == 0
        assert ((out[0].double() - want).abs() <= want * (2.0 ** -8 + 128 * 2.0 ** -24 + 2.0 ** -17)).all()
