"""The marked contexts of marked_cases.py: a tile, or a run of tiles, that is lost, doubled or of another place is
outside the tolerance of every row that sees it, at the lengths at which the GPU tests use them."""
import numpy as np
import pytest

from oracle import window as plain
from tests.marked_cases import SCALE, queries, rows, tolerance

# tokens, rows, dims, window, sinks: those of test_gpu_marked.py
SHAPES = [(20011, 3, 128, None, 0), (9000, 70, 64, None, 0), (7000, 1, 64, None, 0), (9000, 70, 128, 5000, 300),
          (9000, 1, 128, 8000, 20), (30011, 1, 64, 4097, 5), (30011, 1, 128, 30011, 0), (5001, 6, 128, None, 0),
          (2999, 3, 64, 2000, 300)]


def _parts(m, n, window, sinks, d):
    """Numerators [m, heads, tiles, d] and denominators [m, heads, tiles] of every tile, in fp64."""
    k, v = rows(np.arange(n), 1, d)
    q = queries(m, 4, d)
    seen = plain.seen(n, m, window, sinks)
    w = np.exp(SCALE * q[:, :, 0, None] * k[0, None, None, :, 0]) * seen[:, None]
    tiles = -(-n // 64)
    den = np.stack([w[..., 64 * i:64 * i + 64].sum(-1) for i in range(tiles)], -1)
    return den, seen, tiles


@pytest.mark.parametrize("q_type,kv_type", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp4"), ("f32", "f32")])
@pytest.mark.parametrize("n,m,d,window,sinks", SHAPES)
def test_a_lost_or_doubled_tile_is_seen(n, m, d, window, sinks, q_type, kv_type):
    den, seen, tiles = _parts(m, n, window, sinks, d)
    dim = np.arange(tiles) % d
    num = np.stack([den[..., dim == j].sum(-1) for j in range(d)], -1) * 1.5
    total = den.sum(-1)
    ref = num / total[..., None]
    want = plain.attention(queries(m, 4, d), *rows(np.arange(n), 1, d), SCALE, window, sinks)
    assert np.abs(ref - want).max() < 1e-12
    tol = tolerance(ref, q_type, kv_type)
    for i in range(tiles):
        full = seen[:, 64 * i:64 * i + 64].sum(-1) >= 8        # rows that see eight of its tokens or more
        for times in (-1, 1):
            got = num.copy()
            got[..., dim[i]] += times * 1.5 * den[..., i]
            got /= (total + times * den[..., i])[..., None]
            assert (np.abs(got - ref) > tol).any(-1)[full].all(), (i, times)
    # a run of eight tiles lost, and one taken twice in place of its neighbour
    for i in range(0, tiles - 8, 5):
        cut = slice(i, i + 8)
        full = seen[:, 64 * i:64 * i + 512].sum(-1) >= 64
        got = num.copy()
        for j in range(i, i + 8):
            got[..., dim[j]] -= 1.5 * den[..., j]
        got /= (total - den[..., cut].sum(-1))[..., None]
        assert (np.abs(got - ref) > tol).any(-1)[full].all()
        both = (seen[:, 64 * i:64 * i + 128]).all(-1)
        got = num.copy()
        got[..., dim[i]] += 1.5 * den[..., i]
        got[..., dim[i + 1]] -= 1.5 * den[..., i + 1]
        got /= (total + den[..., i] - den[..., i + 1])[..., None]
        assert (np.abs(got - ref) > tol).any(-1)[both].all()


def test_the_references_of_long_contexts_are_blind_without_marks():
    """What the marks are for: with normal values a zero output is within bf16's worst case at 20,011 tokens."""
    from tests.window_cases import bound
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal(s) for s in ((1, 4, 128), (1, 20011, 128), (1, 20011, 128)))
    ref = plain.attention(q, k, v, 128 ** -0.5)
    assert (np.abs(ref) <= bound(q, k, v, 128 ** -0.5, 2.0 ** -8, ref, "bf16")).mean() > 0.99
