"""The 4-bit cache on the GPU: writes bit-exact against the oracle, reads exact, decode
attention within derived bounds of fp64, copies and swaps of its blocks."""
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


def f64(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def cache_of(rng, nb, h, B, d, kv_scale, spread=32.0):
    """A cache of quantised normal rows, as bytes (host) and on the GPU."""
    c = np.zeros(fp4.cache_shape(nb, h, B, d), np.uint8)
    x = (rng.standard_normal((nb * B, h, d)) * spread * kv_scale).astype(np.float32)
    fp4.write(x, c, np.arange(nb * B), kv_scale)
    return c, torch.from_numpy(c).cuda()


# ------------------------------------------------------------------ writes --

@pytest.mark.parametrize("src,d,B,h,kv", [("bf16", 128, 16, 8, 1.0), ("f16", 64, 8, 3, 0.02),
                                          ("f32", 128, 32, 1, 1.7), ("bf16", 64, 32, 5, 2.0 ** -5),
                                          ("f32", 64, 8, 2, 1e-3)])
def test_write_is_bit_exact(src, d, B, h, kv):
    rng = np.random.default_rng(d + B + h)
    nb = 11
    T = min(nb * B - 3, 97)
    x = [torch.from_numpy(rng.standard_normal((T, h, d)).astype(np.float32) *
                          np.float32(10.0 ** rng.uniform(-3, 2, (T, h, 1)))).to(DT[src])
         for _ in range(2)]
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    want = [np.full(fp4.cache_shape(nb, h, B, d), 0xA5, np.uint8) for _ in range(2)]
    got = [torch.from_numpy(w.copy()).cuda() for w in want]
    for w, y in zip(want, x):
        fp4.write(y.float().numpy(), w, slots, kv)
    binding.pkv_reshape_and_cache(x[0].cuda(), x[1].cuda(), got[0], got[1],
                                  torch.from_numpy(slots).cuda(), kv_scale=kv)
    assert binding.pkv_get_device_status() == 0
    for w, g in zip(want, got):
        assert (g.cpu().numpy() == w).all()


def test_write_edges_bit_exact():
    """Ties of codes and scales, zeros, subnormals, saturation, infinities and NaN."""
    d, B = 64, 8
    rows = []
    mids = (fp4.E2M1[1:] + fp4.E2M1[:-1]) / 2
    for s in (1.0, 1.125, 0.0625, 2.0 ** -9):
        g = np.zeros(d, np.float32)
        for i in range(0, d, 16):
            g[i] = 6 * s
            m = np.float32(mids * s)
            g[i + 1:i + 8] = m
            g[i + 8:i + 15] = -np.nextafter(m, np.float32(np.inf if i % 32 else 0))
        rows.append(g)
    smids = (fp4.E4M3[1:] + fp4.E4M3[:-1]) / 2            # scales' midpoints, and neighbours
    for a in np.concatenate([smids, np.nextafter(smids.astype(np.float32), np.float32(0)),
                             np.nextafter(smids.astype(np.float32), np.float32(1e9))]):
        g = np.zeros(d, np.float32)
        g[[0, 17, 34, 51]] = np.float32(a) * 6
        g[[1, 18, 35, 52]] = -np.float32(a)
        rows.append(g)
    for v in (0.0, -0.0, 1e-30, -1e-42, 3e38, np.inf, -np.inf, np.nan):
        g = np.linspace(-1, 1, d).astype(np.float32)
        g[[3, 40]] = v
        rows.append(g)
    x = np.stack(rows)[:, None].astype(np.float32)
    T = x.shape[0]
    nb = -(-T // B)
    for kv in (1.0, 0.37):
        want = np.zeros(fp4.cache_shape(nb, 1, B, d), np.uint8)
        fp4.write(x, want, np.arange(T), kv)
        got = torch.zeros(want.shape, dtype=torch.uint8, device="cuda")
        other = torch.zeros_like(got)
        xt = torch.from_numpy(x).cuda()
        binding.pkv_reshape_and_cache(xt, xt, got, other, torch.arange(T, device="cuda"), kv_scale=kv)
        assert (got.cpu().numpy() == want).all() and torch.equal(got, other)


@pytest.mark.parametrize("src,kv", [("f32", 0.37), ("bf16", 1.0), ("f32", 1e30), ("f16", 3e-36)])
def test_write_rounds_true_quotients(src, kv):
    """Four million codes against IEEE divisions: groups of every magnitude, values on and next
    to the codes' borders for the group's own step."""
    g = torch.Generator("cuda").manual_seed(3)
    T, h, d, B = 4096, 8, 128, 16
    x = torch.randn(T, h, d // 16, 16, generator=g, device="cuda")
    x = x * 2.0 ** torch.randint(-6, 7, (T, h, d // 16, 1), generator=g, device="cuda") * min(kv, 1e28)
    kvt = torch.tensor(kv, device="cuda")

    def step_of(x):
        s = (x.abs().amax(-1) / (6 * kvt)).clamp(max=448.0).to(torch.float8_e4m3fn)
        return s, (s.float() * kvt).unsqueeze(-1)

    x = x.to(DT[src]).float()
    border = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    near = step_of(x)[1] * border * (1 + torch.randint(-2, 3, (T, h, d // 16, 7), generator=g, device="cuda") * 2.0 ** -23)
    x[..., 4:11] = torch.minimum(near, x[..., :4].abs().amax(-1, keepdim=True)) * torch.sign(x[..., 4:11])
    x = x.to(DT[src])
    s, step = step_of(x.float())
    q = torch.where(step > 0, x.float() / step, torch.zeros_like(step))
    m = q.abs()
    code = (m > .25).int() + (m >= .75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
    code = torch.where(step > 0, code + 8 * torch.signbit(q), 0)
    c = torch.zeros(fp4.cache_shape(T // B, h, B, d), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(c)
    x = x.flatten(2)
    binding.pkv_reshape_and_cache(x, x, c, v, torch.arange(T, device="cuda"), kv_scale=kv)
    flat = c.view(T // B, h, -1)
    body = flat[..., :B * d // 2].view(T // B, h, d // 32, B, 16).permute(0, 3, 1, 2, 4).reshape(T, h, d // 2)
    assert torch.equal(torch.stack([body & 15, body >> 4], -1).flatten(-2).int(), code.flatten(2).int())
    sc = flat[..., B * d // 2:].view(T // B, h, B, d // 16).transpose(1, 2).reshape(T, h, -1)
    assert torch.equal(sc, s.view(torch.uint8)) and torch.equal(c, v)


def test_write_flags_slots_outside_and_leaves_the_rest():
    h, d, B, nb = 2, 64, 16, 3
    x = torch.randn(4, h, d, device="cuda")
    c = torch.full(binding.fp4_cache_shape(nb, h, B, d), 0x5A, dtype=torch.uint8, device="cuda")
    v = c.clone()
    slots = torch.tensor([1, nb * B, -7, 20], device="cuda")
    binding.pkv_reshape_and_cache(x, x, c, v, slots)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_SLOT
    want = np.full(c.shape, 0x5A, np.uint8)
    fp4.write(x.cpu().numpy(), want, np.array([1, -1, -1, 20]), 1.0)
    assert (c.cpu().numpy() == want).all() and (v.cpu().numpy() == want).all()


# ------------------------------------------------------------- copy and swap --

@pytest.mark.parametrize("d,B", [(64, 8), (128, 16)])
def test_copy_and_swap_move_whole_tiles(d, B):
    rng = np.random.default_rng(5)
    h, nb = 3, 9
    shape = fp4.cache_shape(nb, h, B, d)
    k, v = (rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
    gk, gv = torch.from_numpy(k.copy()).cuda(), torch.from_numpy(v.copy()).cuda()
    binding.pkv_copy_blocks(gk, gv, [[0, 4], [7, 8]])
    for c in (k, v):
        c[4], c[8] = c[0], c[7]
    assert (gk.cpu().numpy() == k).all() and (gv.cpu().numpy() == v).all()
    hk, hv = (torch.zeros(shape, dtype=torch.uint8).pin_memory() for _ in range(2))
    binding.pkv_swap_blocks(gk, gv, hk, hv, [[8, 0], [2, 5]])
    torch.cuda.synchronize()
    want = np.zeros(shape, np.uint8)
    want[0], want[5] = k[8], k[2]
    assert (hk.numpy() == want).all() and binding.pkv_get_device_status() == 0


# ------------------------------------------------------------------- gather --

def tables_of(rng, lens, B, extra=2):
    need = [-(-n // B) for n in lens]
    nb = sum(need) + extra
    perm = rng.permutation(nb).astype(np.int32)
    t = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = perm[at:at + n]
        at += n
    return t, nb


def rows_of(vals, table, n, B, start=0):
    """[n, h, d] rows start .. start + n - 1 of one sequence from pool values [nb, h, B, d]."""
    tok = np.arange(start, start + n)
    return vals[table[tok // B], :, tok % B]


@pytest.mark.parametrize("d,B,h,out,kv", [(128, 16, 8, "bf16", 0.03125), (64, 8, 1, "f16", 0.02),
                                          (128, 32, 3, "f32", 1.7), (64, 32, 5, "bf16", 1.0),
                                          (128, 8, 2, "f16", 1.0)])
def test_gather_4_bit(d, B, h, out, kv):
    rng = np.random.default_rng(d * B + h)
    lens = [1, 0, 37, B, 0, 100, 3 * B - 1]
    start = [0, 5, 0, 3, 0, 11, 1]
    table, nb = tables_of(rng, [a + b for a, b in zip(lens, start)], B)
    ck, gk = cache_of(rng, nb, h, B, d, kv)
    cv, gv = cache_of(rng, nb, h, B, d, kv)
    row_start = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int32)
    total = int(row_start[-1]) + 5
    ko = torch.full((total, h, d), 7.0, dtype=DT[out], device="cuda")
    vo = torch.full_like(ko, -7.0)
    t = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    r = binding.pkv_gather_cache(gk, gv, t(table), t(row_start), total, DT[out], kv_scale=kv,
                                 token_start=t(start), key_out=ko, value_out=vo)
    assert r[0] is ko and binding.pkv_get_device_status() == 0
    for got, c, fill in ((ko, ck, 7.0), (vo, cv, -7.0)):
        vals = fp4.values(c, d, 1.0)                      # code * scale: exact in fp32
        want = torch.full((total, h, d), fill, dtype=DT[out])
        for s, n in enumerate(lens):
            rows = rows_of(vals, table[s], n, B, start[s])
            y = torch.from_numpy(rows.astype(np.float32)) * torch.tensor(kv, dtype=torch.float32)
            want[row_start[s]:row_start[s + 1]] = y.to(DT[out])
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("kt,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                    ("e4m3", "f32"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("d", [64, 128])
def test_gather_inverts_the_write_for_every_cache(kt, out, d):
    rng = np.random.default_rng(8)
    h, B, T, kv = 3, 16, 75, 0.5 if kt == "e4m3" else 1.0
    table, nb = tables_of(rng, [T], B)
    src = DT[out if kt == "e4m3" else kt]
    x, y = (torch.randn(T, h, d, dtype=torch.float32).to(src) for _ in range(2))
    cdt = torch.float8_e4m3fn if kt == "e4m3" else src
    c, v = (torch.zeros(nb, h, B, d, dtype=torch.uint8 if kt == "e4m3" else cdt, device="cuda").view(cdt)
            for _ in range(2))
    tok = np.arange(T)
    slots = torch.from_numpy(table[0][tok // B].astype(np.int64) * B + tok % B).cuda()
    binding.pkv_reshape_and_cache(x.cuda(), y.cuda(), c, v, slots, kv_scale=kv)
    rs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    k2, v2 = binding.pkv_gather_cache(c, v, torch.from_numpy(table).cuda(), rs, T, DT[out], kv_scale=kv)
    for a, b in ((x, k2), (y, v2)):
        if kt == "e4m3":
            a = ((a.float() / kv).to(torch.float8_e4m3fn).float() * kv).to(DT[out])
        assert torch.equal(b.cpu(), a)
    assert binding.pkv_get_device_status() == 0


def test_gather_skips_and_flags_bad_places():
    rng = np.random.default_rng(9)
    h, B, d, nb = 2, 16, 64, 4
    c, g = cache_of(rng, nb, h, B, d, 1.0)
    table = torch.tensor([[1, nb, 2], [-5, 3, 0]], dtype=torch.int32, device="cuda")
    rs = torch.tensor([0, 48, 60], dtype=torch.int32, device="cuda")
    ko = torch.full((60, h, d), 9.0, dtype=torch.float16, device="cuda")
    binding.pkv_gather_cache(g, g, table, rs, 60, torch.float16, key_out=ko)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_BLOCK_ID
    vals = fp4.values(c, d, 1.0)
    want = np.full((60, h, d), 9.0)
    want[:16] = vals[1].transpose(1, 0, 2)
    want[32:48] = vals[2].transpose(1, 0, 2)
    assert (f64(ko) == want).all()                        # rows of blocks nb and -5 untouched
    for ts in ([40, 0], [-1, 16]):                        # runs over the table's end, or before it
        ko.fill_(9.0)
        binding.pkv_gather_cache(g, g, torch.tensor([[1, 2, 3]] * 2, dtype=torch.int32, device="cuda"),
                                 torch.tensor([0, 20, 20], dtype=torch.int32, device="cuda"), 60,
                                 torch.float16, key_out=ko,
                                 token_start=torch.tensor(ts, dtype=torch.int32, device="cuda"))
        assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
        tok = ts[0] + np.arange(20)
        ok = (tok >= 0) & (tok < 48)
        want[...] = 9.0
        want[:20][ok] = vals[np.array([1, 2, 3])[tok[ok] // B], :, tok[ok] % B]
        assert (f64(ko) == want).all()


# ------------------------------------------------------------------- decode --

def decode_bound(q, rows_k, rows_v, scale, dt):
    """How far a decode output may be from fp64 (per element, rows [h, n, d]).

    Weights p are held in 16 bits with half a step 2^-11 relative (two terms, 2^-22, for fp32
    queries) in numerator and denominator; logits are fp32 sums over d terms, off by at most
    (d + 8) 2^-24 sum |q k| scale, which moves a weight by that much relatively (twice: against
    the maximum), and a weight's exponential by 2^-21; the sums over n tokens are fp32, in runs
    merged by rescaling: (n / 16 + 32) 2^-24 at the very most of sum p |v|; then one rounding."""
    h, n, d = rows_k.shape
    g = q.shape[0] // h
    z = np.einsum("hgd,hnd->hgn", np.abs(q).reshape(h, g, d), np.abs(rows_k)).max(-1) * scale
    ep = 2.0 ** -22 if dt == "f32" else 2.0 ** -11
    rel = 2 * ep + 4 * (d + 8) * 2.0 ** -24 * z + 2.0 ** -19 + 2 * (n / 16 + 32) * 2.0 ** -24
    vmax = np.abs(rows_v).max(1)                          # [h, d]
    return (rel[..., None] * vmax[:, None]).reshape(-1, d)


def check_decode(rng, lens, hq, h, d, B, dt, kv, prefix=False, q_mul=1.0, ctx=None, max_ctx=None):
    table, nb = tables_of(rng, lens, B)
    ck, gk = cache_of(rng, nb, h, B, d, kv)
    cv, gv = cache_of(rng, nb, h, B, d, kv)
    # rows beyond a context hold NaN scales
    used = np.zeros((nb, B), bool)
    for s, n in enumerate(lens):
        tok = np.arange(n)
        used[table[s][tok // B], tok % B] = True
    for c, g in ((ck, gk), (cv, gv)):
        sc = fp4._split(c, d)[1]
        sc[(~used)[:, None, :].repeat(h, 1)] = 0x7F
        g.copy_(torch.from_numpy(c))
    S = len(lens)
    q = (torch.from_numpy(rng.standard_normal((S, hq, d))) * (q_mul / (32 * kv))).to(DT[dt])
    scale = 1 / math.sqrt(d)
    max_ctx = max(max(lens), 1) if max_ctx is None else max_ctx
    if max_ctx > table.shape[1] * B:
        pad = np.full((S, -(-max_ctx // B) - table.shape[1]), -1, np.int32)
        table = np.concatenate([table, pad], 1)
    out = torch.full((S, hq, d), float("nan"), dtype=DT[dt], device="cuda")
    cl = torch.tensor(lens if ctx is None else ctx, dtype=torch.int32, device="cuda")
    args = (q.cuda(), gk, gv, torch.from_numpy(table).cuda(), cl, max_ctx, scale)
    binding.pkv_paged_decode_attention(*args, kv_scale=kv, out=out, prefix=prefix)
    assert binding.pkv_get_device_status() == 0
    vk, vv = fp4.values(ck, d, kv), fp4.values(cv, d, kv)
    for s, n in enumerate(lens):
        rk, rv = (rows_of(x, table[s], n, B).transpose(1, 0, 2) for x in (vk, vv))
        ref = fp4.attention(f64(q[s]), rk, rv, scale)
        got = f64(out[s])
        if n == 0:
            assert (got == 0).all()
            continue
        tol = decode_bound(f64(q[s]), rk, rv, scale, dt) * (1 + HALF[dt]) + HALF[dt] * np.abs(ref)
        assert np.isfinite(got).all()
        err = np.abs(got - ref)
        assert (err <= tol + 1e-30).all(), (s, n, float((err / (tol + 1e-30)).max()))
    return args, out


@pytest.mark.parametrize("hq,h,d,B,dt,kv", [
    (8, 2, 128, 16, "bf16", 1.0), (4, 4, 64, 8, "f16", 0.02), (14, 2, 128, 32, "f16", 1.7),
    (16, 2, 64, 16, "bf16", 2.0 ** -5), (9, 1, 128, 8, "bf16", 1.0), (24, 2, 64, 32, "f16", 1.0),
    (6, 3, 128, 16, "f32", 1.0), (20, 1, 64, 8, "f32", 0.02), (64, 2, 128, 16, "bf16", 1.0),
])
def test_decode_lengths(hq, h, d, B, dt, kv):
    """Empty contexts, single tokens, ends inside and at blocks and tiles, a longer one."""
    check_decode(np.random.default_rng(hq + d + B),
                 [0, 1, B - 1, B, B + 1, 63, 64, 65, 0, 127, 130, 517, 2], hq, h, d, B, dt, kv)


FEW = [(8, 1, 128, 16, "bf16"), (4, 4, 64, 8, "f16"), (12, 1, 128, 32, "f32"), (40, 2, 64, 32, "bf16"),
       (7, 1, 64, 16, "f32"), (32, 2, 128, 8, "f16")]


@pytest.mark.parametrize("lens", [[128, 0, 1, 77], [256, 129, 0, 5], [0, 512, 257, 128], [0, 1, 127, 129, 1025, 700]])
@pytest.mark.parametrize("hq,h,d,B,dt", FEW)
def test_decode_clusters_of_every_size(hq, h, d, B, dt, lens):
    """One, two, four and eight CTAs a unit, with units that leave some of them nothing."""
    check_decode(np.random.default_rng(hq + d + B + len(lens)), lens, hq, h, d, B, dt, 1.0)


@pytest.mark.parametrize("max_ctx", [8192, 8193])
@pytest.mark.parametrize("hq,h,d,B,dt", FEW)
def test_decode_few_sequences_either_way(hq, h, d, B, dt, max_ctx):
    """A bound of the lengths up to 8,192 keeps the clusters, a higher one deals equal runs."""
    check_decode(np.random.default_rng(hq + d + B), [0, 1, 127, 129, 1025, 700], hq, h, d, B, dt, 1.0, max_ctx=max_ctx)


@pytest.mark.parametrize("S,h,most", [(60, 1, 2048), (28, 4, 1024), (56, 8, 512), (56, 8, 513), (240, 8, 128)])
def test_decode_units_near_what_is_resident(S, h, most):
    """Cluster sizes by the number of units, up to four tiles a CTA, and the equal runs beyond."""
    rng = np.random.default_rng(S + h)
    lens = rng.integers(0, most + 1, S)
    lens[S // 2] = most
    check_decode(rng, lens.tolist(), 4 * h, h, 64, 16, "bf16", 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[5000], [3000, 1, 4097], [1]])
def test_decode_split_contexts(dt, lens):
    check_decode(np.random.default_rng(len(lens)), lens, 8, 2, 128, 16, dt, 1.0)


@pytest.mark.parametrize("bound", [4096, 100000])
def test_decode_bound_far_above_the_lengths(bound):
    check_decode(np.random.default_rng(5), [300, 0, 77, 2048], 8, 2, 128, 8, "bf16", 1.0, max_ctx=bound)


def test_decode_nothing_cached():
    check_decode(np.random.default_rng(5), [0] * 40, 8, 2, 128, 8, "bf16", 1.0, max_ctx=0)
    check_decode(np.random.default_rng(5), [0] * 40, 8, 2, 64, 16, "f32", 1.0, max_ctx=500)


def test_decode_many_sequences():
    rng = np.random.default_rng(4)
    check_decode(rng, rng.integers(0, 90, 1500).tolist(), 4, 2, 64, 8, "bf16", 1.0)


@pytest.mark.parametrize("q_mul", [30.0, 1e-3, 0.0])
def test_decode_sharp_and_flat_softmax(q_mul):
    check_decode(np.random.default_rng(6), [700, 33, 1], 8, 2, 128, 16, "bf16", 1.0, q_mul=q_mul)


@pytest.mark.parametrize("dt,q_mul,kv", [("bf16", 1e-9, 1e-9), ("bf16", 1e6, 1e5), ("f32", 1e8, 1e7)])
def test_decode_queries_and_scales_far_from_one(dt, q_mul, kv):
    """q beyond fp16's range with a kv_scale that brings the logits back (and the reverse)."""
    check_decode(np.random.default_rng(7), [300, 65], 4, 2, 64, 16, dt, kv, q_mul=1.0)


@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_decode_takes_any_finite_scale(scale):
    """A scale of 0 weighs every token alike; a negative one turns the order around."""
    rng = np.random.default_rng(14)
    h, hq, d, B, lens = 2, 6, 64, 16, [70, 1, 200]
    table, nb = tables_of(rng, lens, B)
    ck, gk = cache_of(rng, nb, h, B, d, 1.0)
    cv, gv = cache_of(rng, nb, h, B, d, 1.0)
    q = (torch.randn(3, hq, d) / 8).half()
    out = binding.pkv_paged_decode_attention(q.cuda(), gk, gv, torch.from_numpy(table).cuda(),
                                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 200, scale)
    vk, vv = fp4.values(ck, d, 1.0), fp4.values(cv, d, 1.0)
    for s, n in enumerate(lens):
        rk, rv = (rows_of(x, table[s], n, B).transpose(1, 0, 2) for x in (vk, vv))
        ref = fp4.attention(f64(q[s]), rk, rv, scale)
        tol = decode_bound(f64(q[s]), rk, rv, abs(scale), "f16") * 1.01 + HALF["f16"] * np.abs(ref)
        assert (np.abs(f64(out[s]) - ref) <= tol).all()


def test_a_query_row_of_nan_or_infinity_stays_alone():
    rng = np.random.default_rng(15)
    h, d, B = 2, 128, 16
    table, nb = tables_of(rng, [300, 17], B)
    _, g = cache_of(rng, nb, h, B, d, 1.0)
    args = (g, g, torch.from_numpy(table).cuda(), torch.tensor([300, 17], dtype=torch.int32, device="cuda"), 300, 0.05)
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        q = torch.randn(2, 8, d, device="cuda").to(dt) / 32
        ref = binding.pkv_paged_decode_attention(q, *args)
        q[0, 1, 3], q[1, 6, 100] = float("nan"), float("inf")
        got = binding.pkv_paged_decode_attention(q, *args)
        assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 6]).all()
        keep = torch.ones(2, 8, dtype=torch.bool)
        keep[0, 1] = keep[1, 6] = False
        assert torch.equal(got[keep], ref[keep])


def test_caches_beyond_32_bits():
    """Blocks on either side of 2 and 4 GB of each cache: written, fused-written, copied, decoded
    and read back."""
    h, d, B = 8, 128, 16
    tile = h * B * 72
    nb = (1 << 32) // tile + 40
    k = torch.empty(binding.fp4_cache_shape(nb, h, B, d), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    lo, hi = (1 << 31) // tile, (1 << 32) // tile
    blocks = [lo - 1, lo, lo + 1, hi - 1, hi, hi + 1, nb - 1, 0]
    T = len(blocks) * B
    slots = torch.tensor([b * B + r for b in blocks for r in range(B)], device="cuda")
    key, val = (torch.randn(T, h, d, device="cuda").bfloat16() for _ in range(2))
    binding.pkv_reshape_and_cache(key, val, k, v, slots)
    # the same tokens in a small cache at blocks 0, 1, ..
    sk = torch.empty(binding.fp4_cache_shape(len(blocks) + 1, h, B, d), dtype=torch.uint8, device="cuda")
    sv = torch.empty_like(sk)
    binding.pkv_reshape_and_cache(key, val, sk, sv, torch.arange(T, device="cuda"))
    for i, b in enumerate(blocks):
        assert torch.equal(k[b], sk[i]) and torch.equal(v[b], sv[i])
    cs = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).cuda()
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    q = torch.randn(1, 16, d, device="cuda").bfloat16()
    qq = q.expand(T, 16, d).contiguous()
    for c in (k, v):
        c[blocks[:3]] = 0
    binding.pkv_qk_norm_rope_and_cache(qq, key, val, cs, pos, k, v, slots)      # no turn, no norm
    for i, b in enumerate(blocks):
        assert torch.equal(k[b], sk[i]) and torch.equal(v[b], sv[i])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    far, near = i32([blocks]), i32([list(range(len(blocks)))])
    a = binding.pkv_paged_decode_attention(q, k, v, far, i32([T - 3]), T, 0.1)
    b = binding.pkv_paged_decode_attention(q, sk, sv, near, i32([T - 3]), T, 0.1)
    assert torch.equal(a, b)
    a = binding.pkv_gather_cache(k, v, far, i32([0, T]), T, torch.bfloat16)
    b = binding.pkv_gather_cache(sk, sv, near, i32([0, T]), T, torch.bfloat16)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    binding.pkv_copy_blocks(k, v, [[hi + 1, 5], [lo, nb - 2]])
    assert torch.equal(k[5], sk[5]) and torch.equal(v[nb - 2], sv[1])
    assert binding.pkv_get_device_status() == 0


def test_prepared_calls_and_two_streams_at_once():
    """The marshalled calls issue the same work; two decodes run beside each other, each with a
    workspace of its own, one of them captured."""
    rng = np.random.default_rng(16)
    args, out = check_decode(rng, [900, 33, 2500], 8, 2, 128, 16, "bf16", 1.0)
    other, out2 = check_decode(rng, [10, 0, 4000, 777], 16, 1, 64, 32, "f16", 0.5)
    got = torch.empty_like(out)
    call = binding.prepare_paged_decode_attention(*args, out=got)
    call()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    need = binding.pkv_decode_workspace_bytes(4, 16, 1, 64, 32, 4000, "e2m1")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got2 = torch.empty_like(out2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.pkv_paged_decode_attention(*other, kv_scale=0.5, workspace=ws, out=got2)
    torch.cuda.synchronize()
    for _ in range(20):
        got.zero_(), got2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graph.replay()
        binding.pkv_paged_decode_attention(*args, out=got, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(got2, out2)
    # a prepared write, and the write on a stream of its own
    T, h, d, B = 40, 2, 64, 8
    key, val = (torch.randn(T, h, d, device="cuda").half() for _ in range(2))
    slots = torch.randperm(48, device="cuda")[:T]
    a, b, c, e = (torch.zeros(binding.fp4_cache_shape(6, h, B, d), dtype=torch.uint8, device="cuda") for _ in range(4))
    binding.pkv_reshape_and_cache(key, val, a, b, slots)
    call = binding.prepare_reshape_and_cache(key, val, c, e, slots)
    call()
    assert torch.equal(a, c) and torch.equal(b, e)
    rows = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    ref = binding.pkv_gather_cache(a, b, table, rows, 40, torch.float32)
    torch.cuda.synchronize()
    again = binding.pkv_gather_cache(a, b, table, rows, 40, torch.float32, stream=s1)
    torch.cuda.synchronize()
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])
    assert binding.pkv_get_device_status() == 0


def test_decode_prefix_entry_is_the_plain_decode():
    args, out = check_decode(np.random.default_rng(8), [100, 700], 8, 2, 128, 16, "bf16", 1.0)
    again = binding.pkv_paged_decode_attention(*args, prefix=True)
    assert torch.equal(out, again)


def test_decode_noalloc_gives_the_same_bits():
    args, out = check_decode(np.random.default_rng(8), [100, 700, 0, 64], 8, 2, 128, 16, "bf16", 1.0)
    assert torch.equal(out, binding.pkv_paged_decode_attention_noalloc(*args))
    # units of 16 heads and a full chip of workers: the static scratch still suffices
    args, out = check_decode(np.random.default_rng(9), [3000, 40, 1500], 64, 4, 128, 8, "f32", 1.0)
    assert torch.equal(out, binding.pkv_paged_decode_attention_noalloc(*args))
    assert binding.pkv_decode_workspace_bytes(300, 128, 8, 128, 16, 131072, "e2m1") <= binding.NOALLOC_SCRATCH_BYTES


def test_decode_is_deterministic_and_replays_in_a_graph():
    args, out = check_decode(np.random.default_rng(10), [3000, 17, 900], 8, 2, 128, 16, "f16", 1.0)
    need = binding.pkv_decode_workspace_bytes(3, 8, 2, 128, 16, 3000, "e2m1")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.pkv_paged_decode_attention(*args, workspace=ws, out=got)
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.pkv_paged_decode_attention(*args, workspace=ws, out=got)
    for fill in (0, 255):                                  # the workspace need not be zeroed
        ws.fill_(fill)
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    # other lengths in the same buffers, replayed
    args[4].copy_(torch.tensor([64, 17, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, binding.pkv_paged_decode_attention(*args))
    assert binding.pkv_get_device_status() == 0


def test_decode_flags_bad_contexts_and_block_ids():
    rng = np.random.default_rng(11)
    h, d, B = 2, 64, 16
    table, nb = tables_of(rng, [64, 64, 64], B)
    _, g = cache_of(rng, nb, h, B, d, 1.0)
    q = torch.randn(3, 4, d, device="cuda").half()
    good = torch.from_numpy(table).cuda()
    call = lambda t, c: binding.pkv_paged_decode_attention(
        q, g, g, t, torch.tensor(c, dtype=torch.int32, device="cuda"), 64, 0.1)
    ref = call(good, [64, 64, 0])
    got = call(good, [64, 9999, -3])                       # clamped to 64 and 0
    assert binding.pkv_get_device_status() == binding.DEV_BAD_CONTEXT
    assert torch.equal(got, ref)
    bad = good.clone()
    bad[1, 2], bad[2, 0] = nb, -1
    got = call(bad, [64, 64, 64])
    assert binding.pkv_get_device_status() == binding.DEV_BAD_BLOCK_ID
    assert torch.equal(got[0], ref[0])


def test_nan_in_a_context_reaches_only_its_outputs():
    rng = np.random.default_rng(12)
    h, d, B = 2, 128, 16
    table, nb = tables_of(rng, [40, 40], B)
    ck, gk = cache_of(rng, nb, h, B, d, 1.0)
    cv, gv = cache_of(rng, nb, h, B, d, 1.0)
    q = torch.randn(2, 8, d, device="cuda").half() * 0.03
    args = (torch.from_numpy(table).cuda(), torch.tensor([40, 40], dtype=torch.int32, device="cuda"), 40, 0.1)
    ref = binding.pkv_paged_decode_attention(q, gk, gv, *args)
    sc = fp4._split(cv, d)[1]
    sc[table[1, 0], 1, 3, 2] = 0x7F                        # dims 32..47 of kv head 1, sequence 1
    got = binding.pkv_paged_decode_attention(q, gk, torch.from_numpy(cv).cuda(), *args)
    hit = torch.zeros_like(ref, dtype=torch.bool)
    hit[1, 4:, 32:48] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], ref[~hit])


# ---------------------------------------------------------- a run of them --

def test_prompt_fork_and_steps_over_a_4_bit_cache():
    """Block manager, fused norm + rotary + write, copy-on-write, decode, read-back: every
    step's outputs against fp64 over what the cache holds."""
    torch.manual_seed(0)
    h, hq, d, B, nb, kv = 2, 8, 128, 16, 64, 1.0 / 16
    shape = binding.fp4_cache_shape(nb, h, B, d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ang = torch.arange(512).double()[:, None] * 10000.0 ** (-torch.arange(64).double() / 64)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    qw, kw = (1 + 0.1 * torch.randn(d, device="cuda") for _ in range(2))
    m = binding.BlockManager(nb, B)
    lens = {0: 37, 1: 70}
    for s, n in lens.items():
        m.add_sequence(s, n)
        table, _ = m.sequence(s)
        slots = torch.tensor([table[t // B] * B + t % B for t in range(n)], device="cuda")
        qkv = torch.randn(n, (hq + 2 * h) * d, device="cuda").bfloat16()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, h * d, h * d], 1))
        binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, torch.arange(n, device="cuda"), kc, vc, slots,
                                           qw, kw, kv_scale=kv)
    m.fork(0, 2)
    for step in range(4):
        slots, pairs, tables, ctx = m.prepare_step([0, 1, 2], max_blocks=8)
        if len(pairs):
            binding.pkv_copy_blocks(kc, vc, pairs)
        qkv = torch.randn(3, (hq + 2 * h) * d, device="cuda").bfloat16()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, h * d, h * d], 1))
        pos = torch.from_numpy(ctx.astype(np.int64) - 1).cuda()
        q = binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, kc, vc, torch.from_numpy(slots).cuda(),
                                               qw, kw, kv_scale=kv)
        tt, cl = torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()
        out = binding.pkv_paged_decode_attention(q, kc, vc, tt, cl, int(ctx.max()), d ** -0.5, kv_scale=kv)
        rs = torch.from_numpy(np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)).cuda()
        rk, rv = binding.pkv_gather_cache(kc, vc, tt, rs, int(ctx.sum()), torch.float32, kv_scale=kv)
        for s in range(3):
            a, b = int(rs[s]), int(rs[s + 1])
            k64, v64 = f64(rk[a:b]).transpose(1, 0, 2), f64(rv[a:b]).transpose(1, 0, 2)
            ref = fp4.attention(f64(q[s]), k64, v64, d ** -0.5)
            tol = decode_bound(f64(q[s]), k64, v64, d ** -0.5, "bf16") * 1.01 + HALF["bf16"] * np.abs(ref)
            assert (np.abs(f64(out[s]) - ref) <= tol).all()
    # sequences 0 and 2 share their prompt's full blocks and differ in their tails
    assert m.refcount(m.sequence(0)[0][0]) == 2
    assert binding.pkv_get_device_status() == 0


def test_chunked_prefill_over_a_4_bit_context():
    """The prefill kernel reads 16-bit pools: a 4-bit context is read back into one first."""
    rng = np.random.default_rng(13)
    h, hq, d, B, n, new = 2, 8, 128, 16, 83, 21
    table, nb = tables_of(rng, [n + new], B)
    _, gk = cache_of(rng, nb, h, B, d, 1.0)
    _, gv = cache_of(rng, nb, h, B, d, 1.0)
    tt = torch.from_numpy(table).cuda()
    rows = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rk, rv = binding.pkv_gather_cache(gk, gv, tt, rows, n, torch.float16)
    rk, rv = (torch.cat([x, torch.randn(new, h, d, device="cuda").half() * 32]) for x in (rk, rv))
    tok = np.arange(n + new)
    slots = torch.from_numpy(table[0][tok // B].astype(np.int64) * B + tok % B).cuda()
    pk, pv = (torch.zeros(nb, h, B, d, dtype=torch.float16, device="cuda") for _ in range(2))
    binding.pkv_reshape_and_cache(rk, rv, pk, pv, slots)
    q = (torch.randn(new, hq, d, device="cuda") / 32).half()
    out = binding.pkv_paged_multi_query_attention(
        q, pk, pv, tt, torch.tensor([n + new], dtype=torch.int32, device="cuda"),
        torch.tensor([0, new], dtype=torch.int32, device="cuda"), n + new, d ** -0.5)
    k64, v64 = f64(rk).transpose(1, 0, 2), f64(rv).transpose(1, 0, 2)
    for i in range(new):
        m = n + i + 1
        ref = fp4.attention(f64(q[i]), k64[:, :m], v64[:, :m], d ** -0.5)
        tol = decode_bound(f64(q[i]), k64[:, :m], v64[:, :m], d ** -0.5, "f16") + HALF["f16"] * np.abs(ref)
        assert (np.abs(f64(out[i]) - ref) <= tol).all()
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("kt", ["e2m1", "bf16"])
def test_workspace_of_a_call_on_a_busy_stream_is_not_reused_before_it_ran(kt):
    """A call allocates its workspace on the current stream and drops it; where it was asked to run
    on another one, the memory stays taken until that stream is through."""
    rng = np.random.default_rng(31)
    args, out = check_decode(rng, [900, 2500], 8, 2, 128, 16, "bf16", 1.0)
    if kt == "bf16":
        pool = torch.randn(args[1].shape[0], 2, 16, 128, device="cuda").bfloat16()
        args = (args[0], pool, pool, *args[3:])
        out = binding.pkv_paged_decode_attention(*args)
    need = binding.pkv_decode_workspace_bytes(2, 8, 2, 128, 16, 2500, kt)
    got, side = torch.zeros_like(out), torch.cuda.Stream()
    torch.cuda.synchronize()

    def held():
        s = torch.cuda.memory_stats()
        return s["active_bytes.all.current"] - s["allocated_bytes.all.current"]

    before = held()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)                  # some 20 ms
    binding.pkv_paged_decode_attention(*args, out=got, stream=side)
    assert held() - before >= need
    trash = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, out) and len(trash) == 8


def test_decode_takes_a_larger_output_and_a_length_as_a_float():
    rng = np.random.default_rng(32)
    args, out = check_decode(rng, [70, 5], 4, 2, 64, 8, "f16", 1.0)
    big = torch.full((3, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    binding.pkv_paged_decode_attention(*args[:5], float(args[5]), args[6], out=big)
    assert torch.equal(big[:2], out) and (big[2] == 7).all()
    with pytest.raises(ValueError):
        binding.pkv_paged_decode_attention(*args, out=big[:1])
    with pytest.raises(ValueError):
        binding.pkv_paged_decode_attention(*args, out=big[:2].float())
    with pytest.raises(ValueError):
        binding.pkv_paged_decode_attention(*args[:5], 1 << 40, args[6])
    assert binding.pkv_get_device_status() == 0
