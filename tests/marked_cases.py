"""Contexts in which every 64-token tile leaves its mark on the output, so that a lost, doubled or
misplaced one cannot stay within the tolerance, however long the context is.

A token's key is (6, 3, 1.5, 0)[t // 64 mod 4] in dim 0, its value 1.5 in dim t // 64 mod head_dim, all else
zero: every type of cache holds these exactly (4 bits: a scale of 1, 1/2 or 1/4 and a code of 6).  A query is 1, -1, 0
or 1/2 in dim 0, by head, and the scale 2/3 ln 2, so that logits are multiples of 1/2 in log2 units.
"""
import numpy as np
import torch

from oracle import fp4, window as plain
from tests.window_cases import DT, HALF

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


class Marked:
    """Paged contexts of marked tokens, all kv heads alike, with what is not seen poisoned and junk in the tables where
    no seen token lives (the attributes are those of window_cases.Paged)."""

    def __init__(self, rng, lens, new, hq, h, d, B, q_type, kv_type, window, sinks):
        self.lens, self.new, self.hq, self.h, self.d = lens, new, hq, h, d
        self.q_type, self.kv_type, self.window, self.sinks = q_type, kv_type, window, sinks
        self.kv_scale, self.scale, self.most = 1.0, SCALE, max(lens)
        seen = [np.flatnonzero(plain.seen(n, m, window, sinks).any(0)) if n and m else np.zeros(0, int)
                for n, m in zip(lens, new)]
        held = [np.unique(t // B) for t in seen]
        nb = sum(map(len, held)) + 2
        perm = rng.permutation(nb).astype(np.int32)
        table = np.array([-1, nb, 2 ** 31 - 1, -2 ** 31])[rng.integers(0, 4, (len(lens), -(-max(lens) // B)))].astype(np.int32)
        # which of the distinct rows every cached row is; behind these the poison
        kind = [np.full((nb, B), 4), np.full((nb, B), d)]
        at = 0
        for s, (t, blocks) in enumerate(zip(seen, held)):
            table[s, blocks] = perm[at:at + len(blocks)]
            at += len(blocks)
            kind[0][table[s, t // B], t % B] = t // 64 % 4
            kind[1][table[s, t // B], t % B] = t // 64 % d
        distinct = [rows(64 * np.arange(n), 1, d)[i][0] for i, n in ((0, 4), (1, d))]
        self.caches = [self._cache(x, torch.from_numpy(k), B) for x, k in zip(distinct, kind)]
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.gtable, self.glens = i32(table), i32(lens)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.gstart = i32(self.start)
        self.q = torch.from_numpy(queries(sum(new), hq, d)).to(DT[q_type]).cuda()

    def _cache(self, x, kind, B):
        n, d = x.shape
        nb = len(kind)
        kind = kind.cuda()
        if self.kv_type != "fp4":
            t = torch.from_numpy(x).to(torch.float8_e4m3fn if self.kv_type == "e4m3" else DT[self.kv_type])
            poison = torch.full((1, d), float("nan")).to(t.dtype)
            t = torch.cat([a.view(torch.uint8) if self.kv_type == "e4m3" else a for a in (t, poison)]).cuda()
            c = t[kind][:, None].expand(nb, self.h, B, d).contiguous()
            return c.view(torch.float8_e4m3fn) if self.kv_type == "e4m3" else c
        # the bytes of the distinct rows: codes [n, d / 32, 16], scales [n, d / 16]
        small = np.zeros(fp4.cache_shape(n, 1, 8, d), np.uint8)
        fp4.write(x[:, None].astype(np.float32), small, np.arange(n) * 8, 1.0)
        assert np.array_equal(fp4.values(small, d, 1.0)[:, 0, 0], x)
        raw = torch.from_numpy(small.reshape(n, -1)).cuda()
        codes = raw[:, :4 * d].view(n, d // 32, 8, 16)[:, :, 0]
        scales = raw[:, 4 * d:].view(n, 8, d // 16)[:, 0]
        codes = torch.cat([codes, torch.full_like(codes[:1], 0x77)])[kind].transpose(1, 2).reshape(nb, -1)
        scales = torch.cat([scales, torch.full_like(scales[:1], 0x7F)])[kind].reshape(nb, -1)
        tile = torch.cat([codes, scales], 1)[:, None].expand(nb, self.h, -1)
        return tile.contiguous().view(fp4.cache_shape(nb, self.h, B, d))

    def check(self, out):
        out = out.double().cpu().numpy()
        known = {}
        for s, (n, m) in enumerate(zip(self.lens, self.new)):
            if not m:
                continue
            if (n, m) not in known:                       # heads are alike but for the four queries
                known[n, m] = plain.attention(queries(m, 4, self.d), *rows(np.arange(n), 1, self.d), SCALE,
                                              self.window, self.sinks)
            ref = known[n, m][:, np.arange(self.hq) % 4]
            got = out[self.start[s]:self.start[s + 1]]
            bad = ~(np.abs(got - ref) <= tolerance(ref, self.q_type, self.kv_type))
            assert not bad.any(), (s, n, m, np.argwhere(bad)[:4].tolist(), bool(np.isnan(got).any()))
