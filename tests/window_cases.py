"""What the tests of windowed and chunked attention share: paged contexts with everything that is
not seen poisoned, and how far an output may be from fp64."""
import numpy as np
import torch

from oracle import fp4, window as plain

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a step of rounding, relative to the value
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def weight_step(q_type, kv_type):
    """Half a step of the softmax weights' type: operands are the cache's 16-bit type, f16 over FP8
    and 4 bits; fp32 queries keep fp32 weights (two f16 terms over 4 bits)."""
    if q_type == "f32":
        return 2.0 ** -22
    return HALF["bf16"] if kv_type == "bf16" else HALF["f16"]


def bound(q, k, v, scale, ep, ref, dt):
    """How far an output may be from fp64: q [m, Hq, d], k / v [h, n, d] of seen rows.

    Weights are held with half a step ep in numerator and denominator, or lose 2^-25 of the running
    maximum each where f16 ends; logits are fp32 sums over d terms, off by at most
    (d + 8) 2^-24 sum |q k| scale, which moves a weight by that much relatively (twice: against the
    maximum); its exponential is off by 2^-21; the sums over n tokens are fp32, in runs of 16 or
    more merged by rescaling: (n / 16 + 32) 2^-24 of sum p |v| at the very most; queries that are
    scaled into f16 lose 2^-24 of a row's largest; then one rounding to the output's type."""
    m, hq, d = q.shape
    h, n, _ = k.shape
    if n == 0:
        return np.zeros(ref.shape)
    z = np.einsum("mhgd,hnd->mhgn", np.abs(q).reshape(m, h, hq // h, d), np.abs(k)).max(-1) * abs(scale)
    zq = np.abs(q).max(-1).reshape(m, h, -1) * np.abs(k).sum(-1).max(-1)[None, :, None] * abs(scale)
    rel = 2 * ep + n * 2.0 ** -25 * (dt != "f32") + 4 * (d + 8) * 2.0 ** -24 * z + 2.0 ** -19 \
        + 2.0 ** -23 * zq + 2 * (n / 16 + 32) * 2.0 ** -24
    vmax = np.abs(v).max(1)                                   # [h, d]
    err = (rel[..., None] * vmax[None, :, None]).reshape(m, hq, d)
    return err * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + 1e-30


class Paged:
    """Sequences of lens tokens, the last new[s] of them queried, in a cache of kv_type whose
    unseen rows are NaN and whose tables hold junk where no seen token lives."""

    def __init__(self, rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks, kv_scale=1.0,
                 spread=1.0, junk=True):
        self.lens, self.new, self.hq, self.h, self.d, self.B = lens, new, hq, h, d, B
        self.q_type, self.kv_type, self.window, self.sinks = q_type, kv_type, window, sinks
        self.kv_scale, self.scale = kv_scale, d ** -0.5
        held = [sorted({int(t) // B for t in np.flatnonzero(plain.seen(n, m, window, sinks).any(0))})
                if n and m else [] for n, m in zip(lens, new)]
        nb = sum(map(len, held)) + 2
        perm = rng.permutation(nb).astype(np.int32)
        width = max(1, max(-(-n // B) for n in lens))
        junk_ids = np.array([-1, nb, 2 ** 31 - 1, -2 ** 31], np.int64)
        table = junk_ids[rng.integers(0, 4, (len(lens), width))].astype(np.int32) if junk else \
            np.full((len(lens), width), int(perm[-1]), np.int32)
        at = 0
        for s, x in enumerate(held):
            table[s, x] = perm[at:at + len(x)]
            at += len(x)
        self.table = table
        # the cache: everything poisoned, then the rows that are seen
        seen = np.zeros((nb, B), bool)
        for s, (n, m) in enumerate(zip(lens, new)):
            if n and m:
                t = np.flatnonzero(plain.seen(n, m, window, sinks).any(0))
                seen[table[s, t // B], t % B] = True
        mul = 32 * kv_scale if kv_type in ("e4m3", "fp4") else 1.0
        self.caches, self.values = [], []
        for _ in range(2):
            x = rng.standard_normal((nb, B, h, d)).astype(np.float32) * np.float32(mul * spread)
            if kv_type == "fp4":
                c = np.zeros(fp4.cache_shape(nb, h, B, d), np.uint8)
                fp4.write(x.reshape(-1, h, d), c, np.arange(nb * B), kv_scale)
                vals = fp4.values(c, d, kv_scale)
                c.reshape(nb, h, -1)[:, :, B * d // 2:].reshape(nb, h, B, -1).transpose(0, 2, 1, 3)[~seen] = 0x7F
                c = torch.from_numpy(c)
            else:
                t = torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3)))
                if kv_type == "e4m3":
                    c = (t / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
                    vals = c.double().numpy() * np.float64(np.float32(kv_scale))
                    raw = c.view(torch.uint8)
                    raw.permute(0, 2, 1, 3)[torch.from_numpy(~seen)] = 0x7F
                else:
                    c = t.to(DT[kv_type])
                    vals = c.double().numpy()
                    c.permute(0, 2, 1, 3)[torch.from_numpy(~seen)] = float("nan")
            self.caches.append(c.cuda())
            self.values.append(vals)
        q = rng.standard_normal((sum(new), hq, d)) / mul
        self.q = torch.from_numpy(q).to(DT[q_type]).cuda()
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.gtable, self.glens = i32(table), i32(lens)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.gstart = i32(self.start)
        self.most = max(lens)

    def rows(self, s):
        """k, v [h, n, d] of the tokens of sequence s that any of its queries sees, and where they are."""
        n, m = self.lens[s], self.new[s]
        t = np.flatnonzero(plain.seen(n, m, self.window, self.sinks).any(0)) if n and m else np.zeros(0, int)
        k, v = (c[self.table[s, t // self.B], :, t % self.B].transpose(1, 0, 2) for c in self.values)
        return k, v, t

    def check(self, out, scale=None):
        out, scale = f64(out), self.scale if scale is None else scale
        q = f64(self.q)
        ep = weight_step(self.q_type, self.kv_type)
        for s, (n, m) in enumerate(zip(self.lens, self.new)):
            if m == 0:
                continue
            k, v, t = self.rows(s)
            rows = slice(self.start[s], self.start[s + 1])
            kk = np.zeros((self.h, n, self.d))
            vv = np.zeros((self.h, n, self.d))
            kk[:, t], vv[:, t] = k, v
            ref = plain.attention(q[rows], kk, vv, scale, self.window, self.sinks)
            err = np.abs(out[rows] - ref)
            tol = bound(q[rows], k, v, scale, ep, ref, self.q_type)
            assert (err <= tol).all(), (s, n, m, float(np.nanmax(err / tol)), bool(np.isnan(out[rows]).any()))
