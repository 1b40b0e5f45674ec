"""Host validation of the windowed decode and the chunk attention: statuses before any device call."""
import pytest

from paged_kv_cache_87_gb300 import binding, build

E = binding


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _window(lib, **kw):
    a = dict(query=1024, k=1024, v=1024, bt=1024, cl=1024, S=4, Hq=8, Hkv=8, d=64, B=16, NB=64, mb=16, mctx=256,
             w=100, sinks=4, scale=0.125, qt=2, kt=2, kvs=1.0, ws=None, wsb=0, out=1024)
    a.update(kw)
    return lib.pkv_paged_decode_attention_window(
        a["query"], a["k"], a["v"], a["bt"], a["cl"], a["S"], a["Hq"], a["Hkv"], a["d"], a["B"], a["NB"], a["mb"],
        a["mctx"], a["w"], a["sinks"], a["scale"], a["qt"], a["kt"], a["kvs"], a["ws"], a["wsb"], a["out"], None)


@pytest.mark.parametrize("types", [dict(qt=2, kt=2), dict(qt=1, kt=4), dict(qt=2, kt=3, d=128),
                                   dict(qt=0, kt=0), dict(qt=1, kt=3), dict(qt=0, kt=4)])
def test_window_host_validation(lib, types):
    f = lambda **kw: _window(lib, **{**types, **kw})
    assert f(query=None) in (E.PKV_ERR_INVALID_ARG,)
    for bad in (dict(w=0), dict(w=-5), dict(sinks=-1), dict(Hkv=3), dict(Hkv=0), dict(kvs=0.0),
                dict(kvs=float("inf")), dict(scale=float("nan")), dict(mctx=257), dict(mctx=-1), dict(S=-1),
                dict(NB=0), dict(mb=0), dict(B=0), dict(query=1024 + 8), dict(out=1024 + 4), dict(cl=1026)):
        assert f(**bad) == E.PKV_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(B=12)):
        assert f(**bad) == E.PKV_ERR_UNSUPPORTED, bad
    assert f(S=0, query=None, k=None) == E.PKV_OK


def test_window_types_and_workspace(lib):
    assert _window(lib, qt=1, kt=2) == E.PKV_ERR_UNSUPPORTED       # f16 queries, bf16 cache
    assert _window(lib, qt=3) == E.PKV_ERR_UNSUPPORTED             # FP8 queries
    assert _window(lib, kt=9) == E.PKV_ERR_INVALID_ARG
    assert _window(lib, NB=2 ** 24) == E.PKV_ERR_UNSUPPORTED       # 2^31 rows of a pool
    need = binding.pkv_decode_window_workspace_bytes
    # none for the one-launch kernel; else by what is seen, not by the context
    for q, kv, d in (("bf16", "bf16", 64), ("f16", "e4m3", 128), ("f16", "e4m3", 64), ("bf16", "e2m1", 128)):
        assert need(4, 8, 8, d, 16, 10 ** 6, 1000, 4, q, kv) == 0
    assert _window(lib, qt=0, kt=0) == E.PKV_ERR_WORKSPACE
    assert _window(lib, qt=0, kt=3) == E.PKV_ERR_WORKSPACE
    for q, kv, d in (("f32", "f32", 64), ("f32", "e4m3", 64), ("f32", "e2m1", 128), ("f16", "e2m1", 128)):
        a, b = (need(4, 8, 8, d, 16, ctx, 5000, 4, q, kv) for ctx in (20000, 10 ** 6))
        assert a == b > 0
        assert (need(4, 8, 8, d, 16, 100, 5000, 4, q, kv) > 0) == ((q, kv) != ("f16", "e2m1"))
    for bad in ((4, 8, 3, 64, 16, 100, 50, 0), (4, 8, 8, 64, 12, 100, 50, 0), (4, 8, 8, 64, 16, 100, 0, 0),
                (4, 8, 8, 64, 16, 100, 5, -1)):
        assert need(*bad, "f32", "f32") == 0


def _chunk(lib, **kw):
    a = dict(query=1024, k=1024, v=1024, bt=1024, cl=1024, qs=1024, S=4, tq=16, Hq=8, Hkv=2, d=128, B=16, NB=64,
             mb=16, mctx=256, w=2 ** 31 - 1, sinks=0, scale=0.088, qt=2, kt=2, kvs=1.0, ws=None, wsb=0, out=1024)
    a.update(kw)
    return lib.pkv_paged_chunk_attention(
        a["query"], a["k"], a["v"], a["bt"], a["cl"], a["qs"], a["S"], a["tq"], a["Hq"], a["Hkv"], a["d"], a["B"],
        a["NB"], a["mb"], a["mctx"], a["w"], a["sinks"], a["scale"], a["qt"], a["kt"], a["kvs"], a["ws"], a["wsb"],
        a["out"], None)


def test_chunk_host_validation(lib):
    f = lambda **kw: _chunk(lib, **kw)
    for bad in (dict(w=0), dict(sinks=-1), dict(Hkv=3), dict(Hkv=0), dict(kvs=0.0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("inf")), dict(mctx=257), dict(mctx=-1), dict(S=-1), dict(tq=-1), dict(NB=0),
                dict(mb=0), dict(B=0), dict(kt=9), dict(qt=9)):
        assert f(**bad) == E.PKV_ERR_INVALID_ARG, bad
    for bad in (dict(qt=0, kt=0), dict(qt=0, kt=3), dict(qt=1), dict(d=96), dict(B=12), dict(Hq=258, Hkv=2),
                dict(NB=2 ** 27), dict(mctx=2 ** 30 + 16, mb=2 ** 27)):
        assert f(**bad) == E.PKV_ERR_UNSUPPORTED, bad
    assert f() == E.PKV_ERR_WORKSPACE and f(ws=4096 + 16, wsb=1 << 30) == E.PKV_ERR_WORKSPACE
    assert f(ws=4096, wsb=100) == E.PKV_ERR_WORKSPACE
    for bad in (dict(query=None), dict(qs=None), dict(qs=1026), dict(query=1032), dict(out=1032)):
        assert f(**bad) == E.PKV_ERR_INVALID_ARG, bad
    assert f(tq=0, query=None) == E.PKV_OK and f(S=0, tq=0) == E.PKV_OK


def test_chunk_workspace_sizes(lib):
    need = binding.pkv_chunk_workspace_bytes
    one = need(1, 1, 8, 2, 128, 100)
    assert 0 < one < 1 << 21
    assert need(4, 4096, 32, 8, 128, 10 ** 6) < 64 << 20          # two states of every CTA, whatever the lengths
    for bad in ((1, 1, 8, 3, 128, 100), (1, 1, 8, 2, 96, 100), (1, 1, 258, 2, 128, 100), (-1, 1, 8, 2, 128, 100),
                (1, 1, 8, 2, 128, 2 ** 30 + 1)):
        assert need(*bad) == 0
