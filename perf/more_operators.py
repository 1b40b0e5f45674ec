"""Cases for attention over a paged cache under a sliding window, and for chunks of new tokens.

window  one query token a sequence, which sees the last `window` tokens of its context and the
        first `sinks`; the cache is of any type, and the blocks between the two may be gone
        (their table entries are -1)
chunk   one to thousands of new tokens a sequence, each seeing what is before it (all of it, or a
        window and sinks), over a cache of 16 bits, FP8 or 4 bits

The token at position p sees token t <= p where t > p - window or t < sinks.  A cache is
[blocks, kv heads, block, head_dim]; FP8 values are decode(code) * kv_scale; a (block, kv head)
tile of the 4-bit cache holds e2m1 codes [head_dim / 32][block][16 bytes] (dim 2i of a byte in the
low nibble), then e4m3 scales [block][head_dim / 16], and a value is code * scale * kv_scale.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WHOLE = 0                       # a case's window that hides nothing


def _binding():
    from paged_kv_cache_87_gb300 import binding
    return binding


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's chat turn under a window: every microsecond of the call is felt
        dict(name="window, one conversation", op="window", seqs=1, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=20000, hi=20000, window=1024, sinks=4, dtype="bf16",
             cache="bf16", kv_scale=1.0),
        # a serving batch of mixed lengths
        dict(name="window, serving batch", op="window", seqs=256, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=64, hi=32768, window=1024, sinks=4, dtype="bf16",
             cache="bf16", kv_scale=1.0),
        # a wide window over long documents in FP8, eight query heads a kv head
        dict(name="window, long documents FP8", op="window", seqs=64, q_heads=64, kv_heads=8,
             head_dim=128, block=32, lo=4096, hi=131072, window=4096, sinks=16, dtype="bf16",
             cache="fp8", kv_scale=0.03125),
        # one query head a kv head, small heads, small blocks, contexts around an odd window
        dict(name="window, small heads, ragged, 4 bits", op="window", seqs=67, q_heads=20, kv_heads=20,
             head_dim=64, block=8, lo=1, hi=4001, window=511, sinks=3, dtype="f16", cache="fp4",
             kv_scale=0.02),
        # a few draft tokens a sequence are verified
        dict(name="chunk, drafts over FP8", op="chunk", seqs=32, q_heads=32, kv_heads=8, head_dim=128,
             block=16, lo=1024, hi=8192, n_lo=5, n_hi=5, window=WHOLE, sinks=0, dtype="bf16",
             cache="fp8", kv_scale=0.03125),
        # one user's next question after a long document
        dict(name="chunk, one question over 4 bits", op="chunk", seqs=1, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=30000, hi=30000, n_lo=37, n_hi=37, window=WHOLE, sinks=0,
             dtype="bf16", cache="fp4", kv_scale=1.0),
        # prompts taken in chunks of 512 tokens
        dict(name="chunk, prompts over FP8", op="chunk", seqs=16, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=0, hi=8192, n_lo=512, n_hi=512, window=WHOLE, sinks=0,
             dtype="bf16", cache="fp8", kv_scale=0.03125),
        # longer chunks over contexts held in 4 bits
        dict(name="chunk, long contexts over 4 bits", op="chunk", seqs=2, q_heads=32, kv_heads=8,
             head_dim=128, block=32, lo=15000, hi=31000, n_lo=1024, n_hi=1024, window=WHOLE, sinks=0,
             dtype="f16", cache="fp4", kv_scale=1.0),
        # whole prompts under a window
        dict(name="chunk, prompts under a window", op="chunk", seqs=4, q_heads=32, kv_heads=8,
             head_dim=128, block=16, lo=0, hi=0, n_lo=4096, n_hi=16384, window=1024, sinks=4,
             dtype="bf16", cache="bf16", kv_scale=1.0),
        # a mixed step: single tokens and odd chunks, seven query heads a kv head, small heads
        dict(name="chunk, mixed step under a window", op="chunk", seqs=23, q_heads=21, kv_heads=3,
             head_dim=64, block=8, lo=1, hi=5000, n_lo=1, n_hi=301, window=333, sinks=5,
             dtype="f16", cache="fp8", kv_scale=0.02),
    ]


def _log_int(rng, lo, hi):
    lo1, hi1 = max(lo, 1), max(hi, 1)
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo1), math.log(hi1 + 0.5))))))


def draw(rng):
    op = rng.choice(["window", "chunk"])
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 20, 40])
    dtype = rng.choice(["bf16", "bf16", "f16"] + (["f32"] if op == "window" else []))
    cache = rng.choice([dtype, "fp8", "fp4"])
    window = _log_int(rng, 1, 16384)
    case = dict(op=op, head_dim=d, kv_heads=kv_heads, dtype=dtype, cache=cache,
                block=rng.choice([8, 16, 32]), window=window, sinks=rng.choice([0, 0, 1, 4, 5, 16, 130]),
                kv_scale=1.0 if cache == dtype else rng.choice([1.0, 0.03125, 0.02, 1.7]))
    if op == "window":
        case["q_heads"] = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        hi = _log_int(rng, 1, 131072)
        seen = min(hi, window + case["sinks"])
        case.update(lo=_log_int(rng, 1, hi), hi=hi)
        case["seqs"] = _log_int(rng, 1, max(1, min(300, 250_000_000 // (seen * kv_heads * d))))
        return case
    case["q_heads"] = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if rng.random() < 0.5:
        case.update(window=WHOLE, sinks=0)
    n = _log_int(rng, 1, 4096)
    hi = _log_int(rng, 1, 32768)
    seen = min(hi + n, (case["window"] or hi + n) + case["sinks"])
    most = min(250_000_000 // ((hi + n) * kv_heads * d),
               500_000_000_000 // (4 * case["q_heads"] * d * n * seen))
    if most < 1:                        # one short chunk of what is left
        n, most = min(n, 64), 1
        hi = min(hi, 250_000_000 // (kv_heads * d) - n)
    case.update(lo=_log_int(rng, 0, hi), hi=hi, n_lo=_log_int(rng, 1, n), n_hi=n,
                seqs=_log_int(rng, 1, min(64, most)))
    return case


def _spread(case, lo, hi, what):
    """One number a sequence, the same for every seed, spread over [lo, hi] by their logarithm."""
    r = random.Random("%s %d %d %d" % (what, case["seqs"], lo, hi))
    n = [_log_int(r, lo, hi) for _ in range(case["seqs"])]
    n[-1] = hi
    return n


def _new(case):
    """New tokens of each sequence."""
    return [1] * case["seqs"] if case["op"] == "window" else _spread(case, case["n_lo"], case["n_hi"], "new")


def _lens(case):
    """Tokens in the cache of each sequence, the new ones among them."""
    before = _spread(case, case["lo"], case["hi"], "lens")
    return before if case["op"] == "window" else [a + b for a, b in zip(before, _new(case))]


def _seen_tokens(case, n, new):
    """Tokens of a context of n that any of its last `new` tokens sees."""
    if case["window"] == WHOLE:
        return n
    low = max(0, n - new - case["window"] + 1)
    return n - low + min(case["sinks"], low)


def _seen_pairs(case, n, new):
    total = 0
    for p in range(n - new, n):
        low = 0 if case["window"] == WHOLE else max(0, p - case["window"] + 1)
        total += p + 1 - low + min(case["sinks"], low)
    return total


def _row_bytes(case):
    d = case["head_dim"]
    return {"f32": 4 * d, "f16": 2 * d, "bf16": 2 * d, "fp8": d, "fp4": 9 * d / 16}[case["cache"]]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    qd = case["q_heads"] * case["head_dim"]
    lens, new = _lens(case), _new(case)
    tokens = sum(_seen_tokens(case, a, b) for a, b in zip(lens, new))
    pairs = sum(_seen_pairs(case, a, b) for a, b in zip(lens, new))
    return {"bytes": 2 * tokens * case["kv_heads"] * _row_bytes(case) + 2 * sum(new) * qd * e
            + 4 * tokens / case["block"], "flops": 4 * pairs * qd}


# ------------------------------------------------------------------ inputs --

def _fill_fp4(x, kv_scale, block):
    """x [N, h, block, d] in 32 bits -> the bytes of the 4-bit cache that holds it."""
    n, h, b, d = x.shape
    g = x.unflatten(-1, (-1, 16))
    s = (g.abs().amax(-1) / (6 * kv_scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float().unsqueeze(-1) * kv_scale
    a = torch.where(step > 0, g / step, torch.zeros_like(g))
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(a)).to(torch.uint8).view(n, h, b, d // 32, 16, 2)
    code = (code[..., 0] + 16 * code[..., 1]).permute(0, 1, 3, 2, 4).reshape(n, h, -1)
    return torch.cat([code, s.view(torch.uint8).reshape(n, h, -1)], -1).view(n, h, b, 9 * d // 16)


def _pool(gen, case, blocks):
    h, b, d, kind, kv = (case[x] for x in ("kv_heads", "block", "head_dim", "cache", "kv_scale"))
    if kind == "fp4":
        out = torch.empty(blocks, h, b, 9 * d // 16, dtype=torch.uint8, device="cuda")
    else:
        out = torch.empty(blocks, h, b, d, device="cuda",
                          dtype=torch.float8_e4m3fn if kind == "fp8" else DTYPES[kind])
    step = max(1, 2 ** 27 // (h * b * d))
    for i in range(0, blocks, step):
        x = torch.randn(min(step, blocks - i), h, b, d, generator=gen, device="cuda")
        # some channels are several times larger than the rest, as keys' are
        x[..., ::37] *= 5.0
        if kind == "fp8":
            out[i:i + step] = (x * 32).clamp(-448, 448).to(out.dtype)
        elif kind == "fp4":
            out[i:i + step] = _fill_fp4(x * (32 * kv), kv, b)
        else:
            out[i:i + step] = x.to(out.dtype)
    return out


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    lens, new, B = _lens(case), _new(case), case["block"]
    # the blocks that a later token may see are held, those behind the window have been given back
    held = []
    for n, m in zip(lens, new):
        first = 0 if case["window"] == WHOLE else max(0, n - m - case["window"] + 1) // B
        held.append([j for j in range(-(-n // B)) if j >= first or j * B < case["sinks"]])
    blocks = sum(len(x) for x in held) + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], max(1, max(-(-n // B) for n in lens))), -1, dtype=torch.int32)
    row = torch.cat([torch.full((len(x),), s) for s, x in enumerate(held)])
    at = torch.tensor([j for x in held for j in x])
    table = table.cuda()
    table[row.cuda(), at.cuda()] = perm[:blocks - 3]
    st = dict(case)
    quantised = case["cache"] in ("fp8", "fp4")
    # logits of unit spread: the values of a quantised pool are 32 * kv_scale times normal ones
    q = torch.randn(sum(new), case["q_heads"], case["head_dim"], generator=gen, device="cuda")
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    st.update(k=_pool(gen, case, blocks), v=_pool(gen, case, blocks), table=table,
              q=(q / (32 * case["kv_scale"] if quantised else 1)).to(DTYPES[case["dtype"]]),
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), most=max(lens),
              start=torch.tensor(start, dtype=torch.int32, device="cuda"),
              scale=1 / math.sqrt(case["head_dim"]), spans=list(zip(start, new, lens)))
    return st


# ------------------------------------------------------------- plain forms --

def _rows(pool, blk, row, st):
    """The values of cached rows (blk, row), any shape of indices: [..., h, d] in 32 bits."""
    if st["cache"] != "fp4":
        if st["cache"] == "fp8":
            return pool.view(torch.uint8)[blk, :, row].view(torch.float8_e4m3fn).float() * st["kv_scale"]
        return pool[blk, :, row].float()
    d, b = st["head_dim"], st["block"]
    n, h = pool.shape[:2]
    flat = pool.view(n, h, -1)
    c = flat[..., :b * d // 2].view(n, h, d // 32, b, 16)[blk, :, :, row]       # [..., h, d / 32, 16]
    s = flat[..., b * d // 2:].view(n, h, b, d // 16)[blk, :, row].view(torch.float8_e4m3fn)
    c = torch.stack([c & 15, c >> 4], -1).flatten(-3)
    x = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=pool.device)[c.int()]
    return (x.unflatten(-1, (-1, 16)) * s.float().unsqueeze(-1) * st["kv_scale"]).flatten(-2)


def _softmax(z):
    p = (z - z.amax(-1, keepdim=True)).exp()
    return p / p.sum(-1, keepdim=True)


def _plain_window(st):
    B, h, n = st["block"], st["kv_heads"], st["lens"].long()
    low = (n - st["window"]).clamp(min=0)
    first = low.clamp(max=st["sinks"])                          # the sinks that the window leaves out
    j = torch.arange(min(st["most"], st["window"] + st["sinks"]), device="cuda")
    t = torch.where(j < first[:, None], j, low[:, None] + j - first[:, None])
    gone = t >= n[:, None]
    t = t.masked_fill(gone, 0)
    blk = torch.gather(st["table"].long(), 1, t // B).clamp(min=0)
    k = _rows(st["k"], blk, t % B, st).transpose(1, 2)          # [S, h, tokens, d]
    z = torch.matmul(st["q"].float().unflatten(1, (h, -1)) * st["scale"], k.transpose(2, 3))
    del k
    p = _softmax(z.masked_fill(gone[:, None, None], -math.inf))
    return torch.matmul(p, _rows(st["v"], blk, t % B, st).transpose(1, 2)).flatten(1, 2).to(st["q"].dtype)


def _plain_chunk(st):
    B, h, out = st["block"], st["kv_heads"], torch.empty_like(st["q"])
    w, sinks = st["window"] or st["most"], st["sinks"]
    for s, (at, m, n) in enumerate(st["spans"]):
        for i in range(0, m, 512):
            e = min(m, i + 512)
            p = torch.arange(n - m + i, n - m + e, device="cuda")
            low = max(0, n - m + i - w + 1)
            t = torch.arange(low, n - m + e, device="cuda")
            if low > 0 and sinks > 0:
                t = torch.cat([torch.arange(min(sinks, low), device="cuda"), t])
            hidden = (t > p[:, None]) | ((t <= p[:, None] - w) & (t >= sinks))
            blk = st["table"][s].long()[t // B].clamp(min=0)
            k = _rows(st["k"], blk, t % B, st).transpose(0, 1)  # [h, tokens, d]
            q = st["q"][at + i:at + e].float().unflatten(1, (h, -1)).permute(1, 2, 0, 3) * st["scale"]
            z = torch.matmul(q, k[:, None].transpose(2, 3))     # [h, group, rows, tokens]
            p = _softmax(z.masked_fill(hidden, -math.inf))
            v = _rows(st["v"], blk, t % B, st).transpose(0, 1)
            out[at + i:at + e] = torch.matmul(p, v[:, None]).permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
    return out


def run(st):
    if not own:
        return _plain_window(st) if st["op"] == "window" else _plain_chunk(st)
    b = _binding()
    if st["op"] == "window":
        return b.pkv_paged_decode_attention_window(
            st["q"], st["k"], st["v"], st["table"], st["lens"], st["most"], st["scale"],
            st["window"], st["sinks"], kv_scale=st["kv_scale"])
    return b.pkv_paged_chunk_attention(
        st["q"], st["k"], st["v"], st["table"], st["lens"], st["start"], st["most"], st["scale"],
        window=st["window"] or None, sinks=st["sinks"], kv_scale=st["kv_scale"])


# --------------------------------------------------------------- in 64 bits --

def _e4m3(b):
    b = b.to(torch.int64)
    e, m = b // 8 % 16, b % 8
    x = torch.where(e == 0, m.double() * 2.0 ** -9, (1 + m.double() / 8) * 2.0 ** (e - 7).double())
    x = torch.where(b % 128 == 127, torch.full_like(x, math.nan), x)
    return torch.where(b >= 128, -x, x)


def _values64(tiles, case):
    """The values of whole tiles [n, h, block, ...], from the bits of the formats: [n, h, block, d]."""
    kv = torch.tensor(case["kv_scale"], dtype=torch.float32).double().item()
    if case["cache"] == "fp8":
        return _e4m3(tiles.view(torch.uint8)) * kv
    if case["cache"] != "fp4":
        return tiles.double()
    (n, h), d, b = tiles.shape[:2], case["head_dim"], case["block"]
    raw = tiles.reshape(n, h, -1)
    body = raw[:, :, :b * d // 2].reshape(n, h, d // 32, b, 16).to(torch.int64)
    code = torch.empty(n, h, b, d // 32, 32, dtype=torch.int64, device=tiles.device)
    code[..., 0::2] = (body % 16).transpose(2, 3)
    code[..., 1::2] = (body // 16).transpose(2, 3)
    code = code.reshape(n, h, b, d)
    e, m = code // 2 % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + m.double() * 0.5) * 2.0 ** (e - 1).double())
    s = _e4m3(raw[:, :, b * d // 2:].reshape(n, h, b, d // 16))
    return torch.where(code >= 8, -mag, mag) * s.repeat_interleave(16, -1) * kv


def exact(case, seed):
    st = prepare(case, seed)
    B, h, d = case["block"], case["kv_heads"], case["head_dim"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    w = case["window"] if case["window"] != WHOLE else 2 ** 40
    for s, (at, m, n) in enumerate(st["spans"]):
        for i in range(0, m, 256):
            rows = range(n - m + i, n - m + min(m, i + 256))
            # whole blocks from the first that a row sees, and those of the sinks
            b0 = max(0, rows[0] - w + 1) // B
            ids = sorted(set(range(b0, rows[-1] // B + 1)) | set(range(min(b0, -(-case["sinks"] // B)))))
            ids = torch.tensor(ids, device="cuda")
            pos = (ids[:, None] * B + torch.arange(B, device="cuda")).flatten()
            phys = st["table"][s][ids].long()
            k, v = (_values64(st[x][phys], case).transpose(0, 1).reshape(h, -1, d) for x in ("k", "v"))
            p = torch.tensor(list(rows), device="cuda")[:, None]
            seen = (pos <= p) & ((pos > p - w) | (pos < case["sinks"]))
            q = st["q"][at + i:at + i + len(rows)].double().reshape(len(rows), h, -1, d)
            z = torch.einsum("rhgd,htd->hgrt", q, k) * st["scale"]
            a = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
            out[at + i:at + i + len(rows)] = torch.einsum("hgrt,htd->rhgd", a, v).reshape(len(rows), -1, d)
    return out
