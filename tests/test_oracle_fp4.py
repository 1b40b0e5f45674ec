"""Pins of the 4-bit format's oracle, and the host-side refusals of its entry points (CPU)."""
import numpy as np
import pytest
import torch

from oracle import fp4
from paged_kv_cache_87_gb300 import binding, build


def test_tables_are_the_two_formats():
    assert fp4.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (fp4.E4M3 == every).all()


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499, 1), (1.25, 2),
                                    (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (5.0001, 7), (6, 7),
                                    (7.9, 7), (1e30, 7)])
def test_e2m1_ties_go_to_even_and_saturate(x, code):
    # a group whose largest magnitude is 6 has scale 1
    g = np.zeros(16, np.float32)
    g[0], g[3], g[4] = 6, x if x <= 6 else 6, -(x if x <= 6 else 6)
    c, s = fp4.encode(g, 1.0)
    assert s.tolist() == [0x38]
    want = code if x <= 6 else 7
    assert c[3] == want and c[4] == want + 8
    assert fp4.nearest(np.array([x]), fp4.E2M1)[0] == code


def test_scale_edges():
    z, s = fp4.encode(np.zeros(16), 1.0)
    assert not z.any() and s[0] == 0
    tiny = np.full(16, 2.0 ** -10 * 6, np.float32)      # quotient 2^-10: a tie to scale 0
    c, s = fp4.encode(tiny, 1.0)
    assert s[0] == 0 and not c.any()
    c, s = fp4.encode(tiny * 1.01, 1.0)                 # just above: the smallest scale, 2^-9
    assert s[0] == 1 and (c == 5).all()                 # 3.03 steps
    inf = np.zeros(16, np.float32)
    inf[2], inf[5] = np.inf, -1e9
    c, s = fp4.encode(inf, 1.0)
    assert s[0] == 0x7E and c[2] == 7 and c[5] == 15 and c[0] == 0
    nan = np.ones(32, np.float32)
    nan[20] = np.nan
    c, s = fp4.encode(nan, 1.0)
    assert s[0] != 0x7F and s[1] == 0x7F and not c[16:].any()


@pytest.mark.parametrize("d,B", [(64, 8), (128, 16), (128, 32)])
def test_write_then_values_round_trips_within_the_step(d, B):
    rng = np.random.default_rng(d + B)
    nb, h, T = 5, 2, 23
    x = rng.standard_normal((T, h, d)).astype(np.float32)
    cache = np.zeros(fp4.cache_shape(nb, h, B, d), np.uint8)
    slots = rng.permutation(nb * B)[:T]
    slots[4] = -1
    fp4.write(x, cache, slots, 0.25)
    v = fp4.values(cache, d, 0.25)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        y = v[s // B, :, s % B].reshape(h, -1, 16)
        g = x[t].reshape(h, -1, 16)
        amax = np.abs(g).max(-1, keepdims=True)
        # half the widest step (4 to 6: 1 scale), the scale within 2^-4 of amax / 6, and
        # saturation when the scale was rounded down
        assert (np.abs(y - g) <= amax / 6 * (1 + 2.0 ** -4) * 1.0001).all()
    codes = fp4._split(cache, d)[0]
    t = int(np.flatnonzero(slots >= 0)[0])
    c, _ = fp4.encode(x[t], 0.25)
    s = slots[t]
    assert codes[s // B, 1, 1, s % B, 3] == c[1, 32 + 6] | (c[1, 32 + 7] << 4)


def test_norm_rope_is_a_rotation_of_unit_rows():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 64))
    ang = rng.random((9, 16)) * 6
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        y = fp4.norm_rope(x, np.ones(64), cs, np.array([0, 3, 8, 8, 1]), 0.0, inter)
        assert np.allclose((y * y).mean(-1), 1)
        back = fp4.norm_rope(y, None, np.concatenate([np.cos(ang), -np.sin(ang)], 1),
                             np.array([0, 3, 8, 8, 1]), 0.0, inter)
        assert np.allclose(back, x / np.sqrt((x * x).mean(-1, keepdims=True)))


# ---------------------------------------------------------------- refusals --

@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


FP4 = binding.PKV_FP4_E2M1


def test_cache_entry_points_take_the_4_bit_type(lib):
    E = binding
    f = lib.pkv_reshape_and_cache
    assert f(None, 16, 16, 16, 16, 3, 8, 128, 16, 64, 2, FP4, 1.0, None) == E.PKV_ERR_INVALID_ARG
    assert f(16, 16, 16, 16, 16, 3, 8, 128, 16, 64, 2, FP4, 0.0, None) == E.PKV_ERR_INVALID_ARG
    assert f(16, 16, 16, 16, 16, 3, 8, 96, 16, 64, 2, FP4, 1.0, None) == E.PKV_ERR_UNSUPPORTED
    assert f(16, 16, 16, 16, 16, 3, 8, 128, 16, 64, FP4, FP4, 1.0, None) == E.PKV_ERR_UNSUPPORTED
    assert f(16, 16, 16, 16, 16, 3, 8, 128, 16, 64, 2, 5, 1.0, None) == E.PKV_ERR_INVALID_ARG
    assert f(None, None, None, None, None, 0, 8, 64, 8, 64, 0, FP4, 1.0, None) == E.PKV_OK
    assert lib.pkv_copy_blocks(None, None, None, 0, 8, 128, 16, 64, FP4, None) == E.PKV_OK
    assert lib.pkv_copy_blocks(16, 16, 16, 2, 8, 128, 16, 64, 5, None) == E.PKV_ERR_INVALID_ARG
    # prefill kernels read 16-bit pools only
    g = lib.pkv_paged_multi_query_attention
    assert g(16, 16, 16, 16, 16, 16, 4, 16, 8, 2, 128, 16, 64, 16, 256, 0.1, 2, FP4, 1.0, None, 0,
             16, None) == E.PKV_ERR_UNSUPPORTED


def _decode(lib, **kw):
    a = dict(query=1024, k=1024, v=1024, bt=1024, cl=1024, S=4, Hq=8, Hkv=8, d=64, B=16, NB=64,
             mb=16, mctx=256, scale=0.125, qt=2, kvs=1.0, ws=None, wsb=0, out=1024)
    a.update(kw)
    return lib.pkv_paged_decode_attention(a["query"], a["k"], a["v"], a["bt"], a["cl"], a["S"],
                                          a["Hq"], a["Hkv"], a["d"], a["B"], a["NB"], a["mb"],
                                          a["mctx"], a["scale"], a["qt"], FP4, a["kvs"], a["ws"],
                                          a["wsb"], a["out"], None)


def test_decode_refusals(lib):
    E = binding
    assert _decode(lib, query=None) == E.PKV_ERR_INVALID_ARG
    assert _decode(lib, d=96) == E.PKV_ERR_UNSUPPORTED
    assert _decode(lib, B=12) == E.PKV_ERR_UNSUPPORTED
    assert _decode(lib, Hkv=3) == E.PKV_ERR_INVALID_ARG
    assert _decode(lib, qt=FP4) == E.PKV_ERR_UNSUPPORTED
    assert _decode(lib, kvs=0.0) == E.PKV_ERR_INVALID_ARG
    assert _decode(lib, mctx=16 * 16 + 1) == E.PKV_ERR_INVALID_ARG
    assert _decode(lib, k=1024 + 8) == E.PKV_ERR_INVALID_ARG
    assert _decode(lib) == E.PKV_ERR_WORKSPACE
    assert _decode(lib, ws=4096 + 16, wsb=1 << 24) == E.PKV_ERR_WORKSPACE
    assert _decode(lib, ws=4096, wsb=16) == E.PKV_ERR_WORKSPACE
    assert _decode(lib, S=0, query=None) == E.PKV_OK
    for d, B in ((64, 8), (128, 32)):
        assert binding.pkv_decode_workspace_bytes(4, 8, 2, d, B, 1000, "e2m1") > 0
    assert binding.pkv_decode_workspace_bytes(4, 8, 3, 64, 8, 1000, "e2m1") == 0
    assert binding.pkv_decode_workspace_bytes(4, 8, 2, 96, 8, 1000, "e2m1") == 0


def _gather(lib, **kw):
    a = dict(k=16, v=16, bt=16, rs=16, ts=None, S=2, rows=9, H=8, d=128, B=16, NB=64, mb=4, kt=FP4,
             kvs=1.0, ot=2, ko=16, vo=16)
    a.update(kw)
    return lib.pkv_gather_cache(a["k"], a["v"], a["bt"], a["rs"], a["ts"], a["S"], a["rows"],
                                a["H"], a["d"], a["B"], a["NB"], a["mb"], a["kt"], a["kvs"],
                                a["ot"], a["ko"], a["vo"], None)


def test_gather_refusals(lib):
    E = binding
    for bad in (dict(k=None), dict(v=None), dict(bt=None), dict(rs=None), dict(ko=None),
                dict(vo=None), dict(S=-1), dict(rows=-1), dict(H=0), dict(NB=0), dict(mb=0),
                dict(kt=7), dict(ot=7), dict(kvs=0.0), dict(kvs=float("nan")), dict(k=8),
                dict(vo=24), dict(rs=18), dict(ts=18)):
        assert _gather(lib, **bad) == E.PKV_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(B=12), dict(ot=3), dict(ot=FP4), dict(kt=2, ot=1),
                dict(kt=1, ot=0)):
        assert _gather(lib, **bad) == E.PKV_ERR_UNSUPPORTED, bad
    assert _gather(lib, S=0, k=None) == E.PKV_OK
    assert _gather(lib, rows=0, k=None) == E.PKV_OK


def _norm(lib, cache=False, **kw):
    a = dict(q=16, qs=4096, k=16, ks=1024, v=16, vs=1024, qw=16, kw=16, wt=2, eps=1e-6, cs=16,
             mp=100, rot=128, il=0, pos=16, T=3, Hq=32, Hkv=8, d=128, dt=2, qo=16, qos=4096, ko=16,
             kos=1024, kc=16, vc=16, sl=16, B=16, NB=64, kt=2, kvs=1.0)
    a.update(kw)
    mid = [a["qw"], a["kw"], a["wt"], a["eps"], a["cs"], a["mp"], a["rot"], a["il"], a["pos"],
           a["T"], a["Hq"], a["Hkv"], a["d"], a["dt"], a["qo"], a["qos"]]
    if cache:
        return lib.pkv_qk_norm_rope_and_cache(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                                              *mid, a["kc"], a["vc"], a["sl"], a["B"], a["NB"],
                                              a["kt"], a["kvs"], None)
    return lib.pkv_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], *mid, a["ko"], a["kos"], None)


def test_norm_rope_refusals(lib):
    E = binding
    both = [dict(q=None), dict(k=None), dict(cs=None), dict(pos=None), dict(qo=None), dict(T=-1),
            dict(Hq=0), dict(Hkv=0), dict(mp=0), dict(rot=0), dict(dt=9), dict(wt=9),
            dict(eps=-1.0), dict(eps=float("inf")), dict(qs=4095), dict(qs=4100), dict(ks=1023),
            dict(ks=1028), dict(qos=4088), dict(qos=4100), dict(q=8), dict(k=8), dict(qw=8),
            dict(kw=8), dict(cs=8), dict(pos=20), dict(qo=8)]
    for cache in (False, True):
        for bad in both:
            assert _norm(lib, cache, **bad) == E.PKV_ERR_INVALID_ARG, (cache, bad)
        for bad in (dict(d=96), dict(rot=24), dict(rot=144), dict(dt=3), dict(dt=FP4), dict(wt=1)):
            assert _norm(lib, cache, **bad) == E.PKV_ERR_UNSUPPORTED, (cache, bad)
        assert _norm(lib, cache, T=0, q=None) == E.PKV_OK
    for bad in (dict(ko=None), dict(ko=8), dict(kos=1016), dict(kos=1028)):
        assert _norm(lib, **bad) == E.PKV_ERR_INVALID_ARG, bad
    for bad in (dict(v=None), dict(v=8), dict(vs=1016), dict(vs=1028), dict(kc=None),
                dict(vc=8), dict(sl=None), dict(sl=12), dict(NB=0), dict(kt=9),
                dict(kt=FP4, kvs=0.0)):
        assert _norm(lib, True, **bad) == E.PKV_ERR_INVALID_ARG, bad
    for bad in (dict(B=12), dict(kt=1)):
        assert _norm(lib, True, **bad) == E.PKV_ERR_UNSUPPORTED, bad


def test_binding_refuses_before_any_call(lib):
    z = torch.zeros
    q, k = z(3, 4, 64, dtype=torch.bfloat16), z(3, 2, 64, dtype=torch.bfloat16)
    cs, pos, slots = z(9, 64), z(3, dtype=torch.int64), z(3, dtype=torch.int64)
    kc = z(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                        # another type of key
        binding.pkv_qk_norm_rope(q, k.half(), cs, pos)
    with pytest.raises(ValueError):                        # CPU tensors
        binding.pkv_qk_norm_rope(q, k, cs, pos)
    with pytest.raises(ValueError):
        binding.pkv_qk_norm_rope(q, k, cs.half(), pos)
    with pytest.raises(ValueError):
        binding.pkv_qk_norm_rope(q, k, cs, pos.int())
    with pytest.raises(ValueError):                        # int32 slots
        binding.pkv_qk_norm_rope_and_cache(q, k, k, cs, pos, kc, kc, slots.int())
    with pytest.raises(ValueError):                        # another head_dim in the cache
        binding.pkv_qk_norm_rope_and_cache(q, k, k, cs, pos, z(4, 2, 16, 128), z(4, 2, 16, 128), slots)
    i32 = lambda *s: z(*s, dtype=torch.int32)
    f4 = z(*binding.fp4_cache_shape(4, 2, 16, 128), dtype=torch.uint8)
    assert f4.shape == (4, 2, 16, 72) and binding._cache_type(f4) == (FP4, 128)
    assert binding._cache_type(z(4, 2, 16, 64, dtype=torch.uint8)) == (binding.PKV_FP8_E4M3, 64)
    with pytest.raises(ValueError):                        # row_start of the wrong length
        binding.pkv_gather_cache(f4, f4, i32(3, 4), i32(3), 5, torch.float16)
    with pytest.raises(ValueError):
        binding.pkv_gather_cache(f4, f4[:, :1], i32(3, 4), i32(4), 5, torch.float16)
    with pytest.raises(ValueError):                        # a negative number of rows
        binding.pkv_gather_cache(f4, f4, i32(3, 4), i32(4), -1, torch.float16)
    with pytest.raises(TypeError):
        binding.pkv_gather_cache(f4, f4, None, i32(4), 5, torch.float16)
    with pytest.raises(KeyError):                          # a type that the library does not know
        binding.pkv_qk_norm_rope(q.double(), k.double(), cs, pos)
    with pytest.raises(ValueError):                        # too few slots
        binding.pkv_reshape_and_cache(k, k, kc, kc, slots[:2])
    with pytest.raises(ValueError):                        # a row of tables for each query
        binding.pkv_paged_decode_attention(z(3, 4, 64, dtype=torch.bfloat16), kc, kc, i32(2, 4), i32(3), 64, 0.1)
    with pytest.raises(ValueError):                        # queries of another head_dim
        binding.pkv_paged_decode_attention(z(1, 2, 64), f4, f4, i32(1, 4), i32(1), 64, 0.1)
