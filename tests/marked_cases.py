"""Contexts in which every 64-token tile leaves its mark on the output, so that a lost, doubled or
misplaced one cannot stay within the tolerance, however long the context is.

A token's key is (6, 3, 1.5, 0)[t // 64 mod 4] in dim 0, its value 1.5 in dim t // 64 mod head_dim, all else
zero: every type of cache holds these exactly (4 bits: a scale of 1, 1/2 or 1/4 and a code of 6).  A query is 1, -1, 0
or 1/2 in dim 0, by head, and the scale 2/3 ln 2, so that logits are multiples of 1/2 in log2 units.
"""
import numpy as np
import torch

from oracle import fp4, window as plain
from tests.window_cases import DT, HALF, Paged

SCALE = float(np.float32(2 / 3 * np.log(2)))
TURN = (1.0, -1.0, 0.0, 0.5)


def rows(t, h, d):
    """k, v [h, len(t), d] of tokens t."""
    tile = np.asarray(t) // 64
    k, v = np.zeros((2, len(tile), d))
    k[:, 0] = np.array([6.0, 3.0, 1.5, 0.0])[tile % 4]
    v[np.arange(len(tile)), tile % d] = 1.5
    return np.repeat(k[None], h, 0), np.repeat(v[None], h, 0)


def queries(m, hq, d):
    q = np.zeros((m, hq, d))
    q[:, :, 0] = np.array(TURN)[np.arange(hq) % 4]
    return q


def tolerance(ref, q_type, kv_type):
    """Logits are multiples j / 2 of log2 units to 2^-21 (one rounding of scale, of the products' sum and of their
    product each, at most 4 large), so weights of whole j are the powers of two in 16 bits and those between are off
    by half a step of the weights' type, alike in all tokens of one key: numerator and denominator are off by that
    much at most; sums of at most 2^15 such terms, each 11 bits in steps of 2^-4 of the largest or more, are off by
    2^-18 where they do not fit 24 bits (32 adds of 16-token sums a run, joined by factors off by 2^-20); then one rounding."""
    step = 2.0 ** -22 if q_type == "f32" else HALF["bf16" if kv_type == "bf16" else "f16"]
    return np.abs(ref) * (2 * step + 2.0 ** -15 + HALF[q_type])


class Marked(Paged):
    """Paged contexts of marked tokens; what is not seen is poisoned as there."""

    def __init__(self, rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks):
        super().__init__(rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks)
        self.scale = SCALE
        nb = self.caches[0].shape[0]
        content = [np.zeros((nb, B, h, d)) for _ in range(2)]
        seen = np.zeros((nb, B), bool)
        for s, (n, m) in enumerate(zip(lens, new)):
            t = np.flatnonzero(plain.seen(n, m, window, sinks).any(0)) if n and m else np.zeros(0, int)
            blk, at = self.table[s, t // B], t % B
            seen[blk, at] = True
            for x, r in zip(content, rows(t, h, d)):
                x[blk, at] = r.transpose(1, 0, 2)
        self.caches = []
        for x in content:
            if kv_type == "fp4":
                c = np.zeros(fp4.cache_shape(nb, h, B, d), np.uint8)
                fp4.write(x.reshape(-1, h, d).astype(np.float32), c, np.arange(nb * B), 1.0)
                assert np.array_equal(fp4.values(c, d, 1.0), x.transpose(0, 2, 1, 3))
                c.reshape(nb, h, -1)[:, :, B * d // 2:].reshape(nb, h, B, -1).transpose(0, 2, 1, 3)[~seen] = 0x7F
                c = torch.from_numpy(c)
            else:
                t = torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3)))
                c = t.to(torch.float8_e4m3fn if kv_type == "e4m3" else DT[kv_type])
                raw = c.view(torch.uint8) if kv_type == "e4m3" else c
                raw.permute(0, 2, 1, 3)[torch.from_numpy(~seen)] = 0x7F if kv_type == "e4m3" else float("nan")
            self.caches.append(c.cuda())
        self.q = torch.from_numpy(queries(sum(new), hq, d)).to(DT[q_type]).cuda()

    def check(self, out):
        out = out.double().cpu().numpy()
        for s, (n, m) in enumerate(zip(self.lens, self.new)):
            if not m:
                continue
            ref = plain.attention(queries(m, self.hq, self.d), *rows(np.arange(n), self.h, self.d), SCALE,
                                  self.window, self.sinks)
            got = out[self.start[s]:self.start[s + 1]]
            bad = ~(np.abs(got - ref) <= tolerance(ref, self.q_type, self.kv_type))
            assert not bad.any(), (s, n, m, np.argwhere(bad)[:4].tolist(), bool(np.isnan(got).any()))
