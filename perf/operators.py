"""Cases for the operators around the 4-bit paged KV cache.

decode      single-query decode attention over a paged cache held in 4 bits
norm        per-head RMS norm of queries and keys with the rotary embedding, one pass
norm_cache  the same pass writing keys and values straight into a paged 16- or 32-bit cache
write_read  new tokens quantised into the 4-bit cache and read back
gather      contexts of the 4-bit cache read back into contiguous rows

A (block, kv head) tile of the 4-bit cache holds e2m1 codes [head_dim / 32][block][16 bytes]
(dim 2i of a byte in the low nibble), then e4m3 scales [block][head_dim / 16]; a value is
code * scale * kv_scale.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
MAX_POSITION = 131072


def _binding():
    from paged_kv_cache_87_gb300 import binding
    return binding


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's chat turn: every microsecond of the call is felt
        dict(name="decode, one short context", op="decode", seqs=1, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=600, hi=600, dtype="bf16", kv_scale=1.0),
        # a serving batch of mixed lengths, four query heads to a kv head
        dict(name="decode, serving batch", op="decode", seqs=256, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=64, hi=8192, dtype="bf16", kv_scale=0.03125),
        # few very long documents: the context is split over the whole chip
        dict(name="decode, long documents", op="decode", seqs=8, q_heads=64, kv_heads=8,
             head_dim=128, block=32, lo=32768, hi=131072, dtype="bf16", kv_scale=1.0),
        # one query head to a kv head, small heads, small blocks, ragged lengths
        dict(name="decode, small heads, ragged", op="decode", seqs=67, q_heads=20, kv_heads=20,
             head_dim=64, block=8, lo=1, hi=4001, dtype="f16", kv_scale=0.02),
        # one decode step's new tokens of a batch
        dict(name="norm and cache, decode step", op="norm_cache", tokens=64, q_heads=32,
             kv_heads=8, head_dim=128, block=16, rot=128, interleaved=False, dtype="bf16"),
        # a batch of prompts
        dict(name="norm and cache, prompts", op="norm_cache", tokens=16384, q_heads=32,
             kv_heads=8, head_dim=128, block=16, rot=128, interleaved=False, dtype="bf16"),
        # a single token
        dict(name="norm, one token", op="norm", tokens=1, q_heads=32, kv_heads=8, head_dim=128,
             rot=128, interleaved=False, dtype="bf16"),
        # an odd number of tokens, half the dims rotated in adjacent pairs
        dict(name="norm, odd chunk", op="norm", tokens=3001, q_heads=40, kv_heads=40,
             head_dim=64, rot=32, interleaved=True, dtype="f16"),
        # one decode step's new tokens
        dict(name="write and read, decode step", op="write_read", tokens=61, kv_heads=8,
             head_dim=128, block=16, dtype="bf16", kv_scale=0.03125),
        # prompts
        dict(name="write and read, prompts", op="write_read", tokens=32768, kv_heads=8,
             head_dim=128, block=16, dtype="bf16", kv_scale=1.0),
        # one context handed to a path that wants 16 bits
        dict(name="gather, one context", op="gather", seqs=1, kv_heads=8, head_dim=128, block=16,
             lo=5000, hi=5000, dtype="bf16", kv_scale=1.0),
        # a batch of contexts
        dict(name="gather, batch", op="gather", seqs=48, kv_heads=8, head_dim=128, block=32,
             lo=100, hi=16384, dtype="f16", kv_scale=0.02),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "norm", "norm_cache", "write_read", "gather"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    block = rng.choice([8, 16, 32])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 20, 40])
    kv_scale = rng.choice([1.0, 0.03125, 0.02, 1.7])
    case = dict(op=op, kv_heads=kv_heads, head_dim=d, dtype=dtype)
    if op in ("decode", "gather"):
        hi = _log_int(rng, 1, 131072 if op == "decode" else 16384)
        lo = _log_int(rng, 1, hi)
        most = (700_000_000 if op == "decode" else 2 ** 26) // (hi * kv_heads * d)
        case.update(seqs=_log_int(rng, 1, max(1, min(300, most))), lo=lo, hi=hi, block=block,
                    kv_scale=kv_scale)
        if op == "decode":
            case["q_heads"] = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    else:
        case["tokens"] = _log_int(rng, 1, 16384)
        if op == "write_read":
            case.update(block=block, kv_scale=kv_scale)
            case["tokens"] = min(case["tokens"], 48_000_000 // (kv_heads * d))
        else:
            case.update(q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), rot=rng.choice([16, 32, d]),
                        interleaved=rng.random() < 0.5)
            most = 90_000_000 // ((case["q_heads"] + 2 * kv_heads) * d)
            case["tokens"] = min(case["tokens"], most)
            if op == "norm_cache":
                case["block"] = block
    return case


def _lens(case):
    """The context lengths: the same for every seed, spread over [lo, hi] by their logarithm."""
    r = random.Random("%d %d %d" % (case["seqs"], case["lo"], case["hi"]))
    n = [_log_int(r, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[-1] = case["hi"]
    return n


def work(case):
    h, d, op = case["kv_heads"], case["head_dim"], case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    row4 = h * d * 9 / 16                         # bytes of a token's keys in the 4-bit cache
    if op == "decode":
        tokens, qd = sum(_lens(case)), case["q_heads"] * d
        tables = sum(-(-n // case["block"]) for n in _lens(case)) * 4
        return {"bytes": 2 * tokens * row4 + 2 * case["seqs"] * qd * e + tables,
                "flops": 4 * tokens * qd}
    if op == "gather":
        tokens = sum(_lens(case))
        return {"bytes": 2 * tokens * (row4 + h * d * e), "flops": 4 * tokens * h * d}
    t = case["tokens"]
    if op == "write_read":
        # the rows are read, their places in the cache and the rows read back are written
        return {"bytes": 2 * t * (2 * h * d * e + row4), "flops": 12 * t * h * d}
    rows = case["q_heads"] + h
    return {"bytes": 2 * t * (rows + (h if op == "norm_cache" else 0)) * d * e
            + min(t, MAX_POSITION) * case["rot"] * 4, "flops": 8 * t * rows * d}


# ------------------------------------------------------------------ inputs --

def _quantise(x, kv_scale):
    """x [..., d] in 32 bits -> (codes 0..15 uint8 [..., d], e4m3 scales [..., d / 16])."""
    g = x.unflatten(-1, (-1, 16))
    kv = torch.tensor(kv_scale, dtype=torch.float32, device=x.device)
    s = (g.abs().amax(-1) / (6 * kv)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s.float() * kv).unsqueeze(-1)
    a = torch.where(step > 0, g / step, torch.zeros_like(g))
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0))
    code = code + 8 * torch.signbit(a)
    return code.to(torch.uint8).flatten(-2), s


def _pack(codes, scales, block):
    """codes [N, h, block, d], scales [N, h, block, d / 16] -> the cache's bytes."""
    n, h, b, d = codes.shape
    c = codes.view(n, h, b, d // 32, 16, 2)
    c = (c[..., 0] + 16 * c[..., 1]).permute(0, 1, 3, 2, 4).reshape(n, h, -1)
    s = scales.view(torch.uint8).reshape(n, h, -1)
    return torch.cat([c, s], -1).view(n, h, b, 9 * d // 16)


def _pool(gen, blocks, h, block, d, kv_scale):
    out = torch.empty(blocks, h, block, 9 * d // 16, dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 27 // (h * block * d))
    for b in range(0, blocks, step):
        x = torch.randn(min(step, blocks - b), h, block, d, generator=gen, device="cuda")
        # some channels are several times larger than the rest, as keys' are
        x[..., ::37] *= 5.0
        out[b:b + step] = _pack(*_quantise(x * (32 * kv_scale), kv_scale), block)
    return out


def _tables(gen, case):
    n = torch.tensor(_lens(case), dtype=torch.int32)
    need = (n + case["block"] - 1) // case["block"]
    blocks = int(need.sum()) + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], int(need.max())), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(int(need.max()))[None, :] < need[:, None]
    table[have.cuda()] = perm[:int(need.sum())]
    return n.cuda(), table, blocks


def _cos_sin(rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, h, d, dt = case["op"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    st = dict(case)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op in ("decode", "gather"):
        n, table, blocks = _tables(gen, case)
        kv = case["kv_scale"]
        st.update(lens=n, table=table, k=_pool(gen, blocks, h, case["block"], d, kv),
                  v=_pool(gen, blocks, h, case["block"], d, kv), most=case["hi"])
        if op == "decode":
            # logits of unit spread: the pool's values are 32 * kv_scale times normal ones
            st["q"] = (rand(case["seqs"], case["q_heads"], d) / (32 * kv)).to(dt)
            st["scale"] = 1 / math.sqrt(d)
        else:
            start = [0]
            for x in _lens(case):
                start.append(start[-1] + x)
            st.update(rows=start[-1], row_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
        return st
    t = case["tokens"]
    if op != "norm":
        blocks = -(-t // case["block"]) + 2
        perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        at = torch.arange(t, device="cuda")
        st["slots"] = perm[at // case["block"]].long() * case["block"] + at % case["block"]
    if op == "write_read":
        st.update(key=rand(t, h, d).to(dt), value=rand(t, h, d).to(dt),
                  table=perm[None, :blocks - 2].contiguous(),
                  row_start=torch.tensor([0, t], dtype=torch.int32, device="cuda"))
        for x in ("k", "v"):
            st[x] = torch.zeros(blocks, h, case["block"], 9 * d // 16, dtype=torch.uint8, device="cuda")
        return st
    # queries, keys and values as one projection leaves them: parts of one row for each token
    hq = case["q_heads"]
    qkv = (3 * rand(t, (hq + 2 * h) * d)).to(dt)
    st.update(q=qkv[:, :hq * d].unflatten(1, (hq, d)),
              key=qkv[:, hq * d:(hq + h) * d].unflatten(1, (h, d)),
              value=qkv[:, (hq + h) * d:].unflatten(1, (h, d)),
              qw=(1 + 0.2 * rand(d)).to(dt), kw=(1 + 0.2 * rand(d)).to(dt),
              cos_sin=_cos_sin(case["rot"]),
              positions=torch.randint(0, MAX_POSITION, (t,), generator=gen, device="cuda"))
    if op == "norm_cache":
        for x in ("k", "v"):
            st[x] = torch.zeros(blocks, h, case["block"], d, dtype=dt, device="cuda")
    return st


# ------------------------------------------------------------- plain forms --

def _unpack(tiles, d, block, kv_scale):
    """tiles [..., h, block, 9 d / 16] -> values [..., h, block, d] in 32 bits."""
    flat = tiles.flatten(-2)
    at = block * d // 2
    c = flat[..., :at].unflatten(-1, (d // 32, block, 16)).transpose(-3, -2)
    c = torch.stack([c & 15, c >> 4], -1).flatten(-3)
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=tiles.device)
    s = flat[..., at:].view(torch.float8_e4m3fn).float().unflatten(-1, (block, d // 16))
    x = lut[c.int()].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)
    return (x * torch.tensor(kv_scale, device=tiles.device)).flatten(-2)


def _context(pool, table, d, block, kv_scale):
    x = _unpack(pool[table.long().clamp(min=0)], d, block, kv_scale)   # [S, blocks, h, block, d]
    return x.transpose(1, 2).flatten(2, 3)                             # [S, h, tokens, d]


def _plain_decode(st):
    d, block, h = st["head_dim"], st["block"], st["kv_heads"]
    k = _context(st["k"], st["table"], d, block, st["kv_scale"])
    q = st["q"].float().unflatten(1, (h, -1)) * st["scale"]
    z = torch.matmul(q, k.transpose(2, 3))
    del k
    past = torch.arange(z.shape[-1], device="cuda") >= st["lens"][:, None]
    z = z.masked_fill(past[:, None, None], -math.inf)
    p = (z - z.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    v = _context(st["v"], st["table"], d, block, st["kv_scale"])
    return torch.matmul(p, v).flatten(1, 2).to(st["q"].dtype)


def _plain_rows(st, dt):
    live = torch.arange(st["table"].shape[1] * st["block"], device="cuda") < st["lens"][:, None]
    return tuple(_context(st[x], st["table"], st["head_dim"], st["block"], st["kv_scale"])
                 .transpose(1, 2)[live].to(dt) for x in ("k", "v"))


def _plain_norm(x, w, st):
    x = x.float()
    x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
    rot = st["rot"]
    cs = st["cos_sin"][st["positions"]][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    if st["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain(st):
    op = st["op"]
    if op == "decode":
        return _plain_decode(st)
    dt = DTYPES[st["dtype"]]
    if op == "gather":
        return _plain_rows(st, dt)
    if op == "write_read":
        got = []
        for x in ("key", "value"):
            c, s = _quantise(st[x].float(), st["kv_scale"])
            pool = st[x[0]]
            n, h, block, _ = pool.shape
            d = st["head_dim"]
            blk, row = st["slots"] // block, st["slots"] % block
            flat = pool.view(n, h, -1)
            pair = c.unflatten(-1, (d // 32, 16, 2))
            code = flat[..., :block * d // 2].view(n, h, d // 32, block, 16)
            code[blk, :, :, row] = pair[..., 0] + 16 * pair[..., 1]
            flat[..., block * d // 2:].view(n, h, block, d // 16)[blk, :, row] = s.view(torch.uint8)
            y = _unpack(pool[blk], d, block, st["kv_scale"])          # [t, h, block, d]
            got.append(y[torch.arange(y.shape[0], device="cuda"), :, row].to(dt))
        return tuple(got)
    q, k = _plain_norm(st["q"], st["qw"], st).to(dt), _plain_norm(st["key"], st["kw"], st).to(dt)
    if op == "norm":
        return q, k
    block = st["block"]
    blk, row = st["slots"] // block, st["slots"] % block
    st["k"][blk, :, row] = k
    st["v"][blk, :, row] = st["value"]
    return q, st["k"], st["v"]


def run(st):
    if not own:
        return _plain(st)
    b, op = _binding(), st["op"]
    if op == "decode":
        return b.pkv_paged_decode_attention(st["q"], st["k"], st["v"], st["table"], st["lens"],
                                            st["most"], st["scale"], kv_scale=st["kv_scale"])
    dt = DTYPES[st["dtype"]]
    if op == "gather":
        return b.pkv_gather_cache(st["k"], st["v"], st["table"], st["row_start"], st["rows"], dt,
                                  kv_scale=st["kv_scale"])
    if op == "write_read":
        b.pkv_reshape_and_cache(st["key"], st["value"], st["k"], st["v"], st["slots"],
                                kv_scale=st["kv_scale"])
        return b.pkv_gather_cache(st["k"], st["v"], st["table"], st["row_start"], st["tokens"], dt,
                                  kv_scale=st["kv_scale"])
    if op == "norm":
        return b.pkv_qk_norm_rope(st["q"], st["key"], st["cos_sin"], st["positions"], st["qw"],
                                  st["kw"], eps=EPS, interleaved=st["interleaved"])
    q = b.pkv_qk_norm_rope_and_cache(st["q"], st["key"], st["value"], st["cos_sin"],
                                     st["positions"], st["k"], st["v"], st["slots"], st["qw"],
                                     st["kw"], eps=EPS, interleaved=st["interleaved"])
    return q, st["k"], st["v"]


# --------------------------------------------------------------- in 64 bits --

def _values64(tiles, d, block, kv_scale):
    """The values of tiles [n, h, block, 9 d / 16], from the bits of the two formats."""
    n, h = tiles.shape[:2]
    raw = tiles.reshape(n, h, -1)
    body = raw[:, :, :block * d // 2].reshape(n, h, d // 32, block, 16).to(torch.int64)
    code = torch.empty(n, h, block, d // 32, 32, dtype=torch.int64, device=tiles.device)
    code[..., 0::2] = (body % 16).transpose(2, 3)
    code[..., 1::2] = (body // 16).transpose(2, 3)
    code = code.reshape(n, h, block, d)
    e, m = code // 2 % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + m.double() * 0.5) * 2.0 ** (e - 1).double())
    x = torch.where(code >= 8, -mag, mag)
    b = raw[:, :, block * d // 2:].reshape(n, h, block, d // 16).to(torch.int64)
    e, m = b // 8 % 16, b % 8
    s = torch.where(e == 0, m.double() * 2.0 ** -9, (1 + m.double() / 8) * 2.0 ** (e - 7).double())
    s = torch.where(b % 128 == 127, torch.full_like(s, math.nan), s)
    s = torch.where(b >= 128, -s, s)
    kv = torch.tensor(kv_scale, dtype=torch.float32).double().item()
    return x * s.repeat_interleave(16, -1) * kv


def _nearest(x, values):
    """Index of the nearest of `values` (0 first, rising) to each x >= 0; a tie goes to the even one."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    mid = (v[1:] + v[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous())
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == x)
    return i + (tie & (i % 2 == 1)).long()


def _exact_quantised(x, kv_scale):
    e4m3 = [m * 2.0 ** -9 for m in range(8)]
    e4m3 += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    kv = torch.tensor(kv_scale, dtype=torch.float32).double().item()
    g = x.double().reshape(*x.shape[:-1], -1, 16)
    table = torch.tensor(e4m3, dtype=torch.float64, device=x.device)
    s = table[_nearest(g.abs().max(-1).values / (6 * kv), e4m3)][..., None] * kv
    mag = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    y = mag[_nearest(torch.where(s > 0, g.abs() / s.clamp(min=1e-300), 0 * g), MAGNITUDES)] * s
    return torch.where(g < 0, -y, y).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["head_dim"]
    if op in ("decode", "gather"):
        block, h, got = case["block"], case["kv_heads"], ([], [])
        for i, n in enumerate(_lens(case)):
            at = st["table"][i, :-(-n // block)].long()
            k, v = (_values64(st[x][at], d, block, case["kv_scale"]).transpose(0, 1).reshape(h, -1, d)[:, :n]
                    for x in ("k", "v"))
            if op == "gather":
                got[0].append(k.transpose(0, 1))
                got[1].append(v.transpose(0, 1))
                continue
            q = st["q"][i].double().reshape(h, -1, d)
            a = torch.softmax(q @ k.transpose(1, 2) * st["scale"], -1)
            got[0].append((a @ v).reshape(-1, d))
        return torch.stack(got[0]) if op == "decode" else (torch.cat(got[0]), torch.cat(got[1]))
    if op == "write_read":
        return tuple(_exact_quantised(st[x], case["kv_scale"]) for x in ("key", "value"))
    rot, t = case["rot"], case["tokens"]

    def turn(x, w):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w.double()
        y = x.clone()
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        cs = st["cos_sin"].double()[st["positions"]].reshape(t, 1, 2, rot // 2)
        z = torch.complex(x[..., a], x[..., b]) * torch.complex(cs[:, :, 0], cs[:, :, 1])
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k = turn(st["q"], st["qw"]), turn(st["key"], st["kw"])
    if op == "norm":
        return q, k
    block = case["block"]
    pools = []
    for rows in (k, st["value"].double()):
        flat = torch.zeros(st["k"].shape[0] * block, *rows.shape[1:], dtype=torch.float64, device="cuda")
        flat[st["slots"]] = rows
        pools.append(flat.reshape(-1, block, *rows.shape[1:]).transpose(1, 2).contiguous())
    return q, pools[0], pools[1]
