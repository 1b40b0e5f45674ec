"""Per-head norm with rotary embedding, alone and with the cache write, against fp64."""
import numpy as np
import pytest
import torch

from oracle import fp4
from paged_kv_cache_87_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.double().cpu().numpy()


def make(T, hq, h, d, rot, dt, wdt, seed=0, max_pos=1000):
    g = torch.Generator().manual_seed(seed)
    qkv = (3 * torch.randn(T, (hq + 2 * h) * d + 16, generator=g)).to(DT[dt]).cuda()
    q, k, v, _ = (qkv.split([hq * d, h * d, h * d, 16], 1))
    q, k, v = (x.unflatten(1, (-1, d)) for x in (q, k, v))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(DT[wdt]).cuda() for _ in range(2)]
    ang = torch.rand(max_pos, rot // 2, generator=g) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda()
    pos = torch.randint(0, max_pos, (T,), generator=g)
    pos[0], pos[-1] = 0, max_pos - 1
    return q, k, v, w, cs, pos.cuda()


def close(got, x, w, cs, pos, eps, inter, dt):
    """|error| <= rounding of the result + fp32 steps before it: the mean square is a sum of d
    squares (d 2^-24 relative at most, halved by the root), root, division and two products add
    8 2^-24, the rotation's two products and sum 3 2^-24 of each term's size."""
    ref = fp4.norm_rope(f64(x), None if w is None else f64(w), f64(cs), pos.cpu().numpy(), eps, inter)
    # |y_i| + |y_j| bounds each rotated value's terms
    y = fp4.norm_rope(f64(x), None if w is None else f64(w), np.concatenate(
        [np.ones((1, cs.shape[1] // 2)), np.zeros((1, cs.shape[1] // 2))], 1), pos.cpu().numpy() * 0, eps, inter)
    r = cs.shape[1]
    size = np.abs(y)
    if inter:
        s = size[..., 0:r:2] + size[..., 1:r:2]
        size[..., 0:r:2] = s
        size[..., 1:r:2] = s
    else:
        s = size[..., :r // 2] + size[..., r // 2:r]
        size[..., :r // 2] = s
        size[..., r // 2:r] = s
    fp32 = (x.shape[-1] / 2 + 11) * 2.0 ** -24 * size
    tol = fp32 * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + 2.0 ** -25 * (dt == "f16")
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())


CASES = [(1, 32, 8, 128, 128, "bf16", "bf16", False), (7, 5, 5, 64, 32, "f16", "f32", True),
         (33, 3, 1, 128, 96, "f32", "f32", False), (19, 40, 40, 64, 64, "bf16", "f32", False),
         (65, 8, 2, 128, 16, "f16", "f16", True), (12, 1, 1, 64, 16, "f32", "f32", True),
         (500, 7, 3, 128, 64, "bf16", "bf16", True), (300, 20, 1, 64, 48, "f16", "f16", False)]


@pytest.mark.parametrize("T,hq,h,d,rot,dt,wdt,inter", CASES)
def test_norm_rope(T, hq, h, d, rot, dt, wdt, inter):
    q, k, _, w, cs, pos = make(T, hq, h, d, rot, dt, wdt)
    qo, ko = binding.pkv_qk_norm_rope(q, k, cs, pos, w[0], w[1], eps=1e-5, interleaved=inter)
    assert binding.pkv_get_device_status() == 0
    close(qo, q, w[0], cs, pos, 1e-5, inter, dt)
    close(ko, k, w[1], cs, pos, 1e-5, inter, dt)
    # without a weight: rotation alone
    qo, k2 = binding.pkv_qk_norm_rope(q, k, cs, pos, None, w[1], eps=1e-5, interleaved=inter)
    close(qo, q, None, cs, pos, 1e-5, inter, dt)
    assert torch.equal(k2, ko)


def test_in_place_on_a_fused_projection_leaves_the_rest():
    T, hq, h, d = 37, 6, 2, 128
    q, k, v, w, cs, pos = make(T, hq, h, d, 64, "bf16", "bf16")
    want = binding.pkv_qk_norm_rope(q, k, cs, pos, *w)
    whole = q._base if q._base is not None else q
    before = whole.clone()
    binding.pkv_qk_norm_rope(q, k, cs, pos, *w, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    tail = slice((hq + h) * d, None)
    assert torch.equal(whole[:, tail], before[:, tail])


@pytest.mark.parametrize("T,hq,h,d,rot,dt,wdt,inter", CASES)
@pytest.mark.parametrize("kt", ["same", "e4m3", "e2m1"])
def test_fused_write_is_the_two_calls_bit_for_bit(T, hq, h, d, rot, dt, wdt, inter, kt):
    B = {64: 8, 128: 16}[d]
    q, k, v, w, cs, pos = make(T, hq, h, d, rot, dt, wdt, seed=1)
    nb, kv = -(-T // B) + 2, 0.05
    rng = np.random.default_rng(T)
    slots = torch.from_numpy(rng.permutation(nb * B)[:T].astype(np.int64))
    slots[T // 2] = -1 if T > 1 else slots[0]
    slots = slots.cuda()
    if kt == "same":
        shape, cdt = (nb, h, B, d), DT[dt]
    else:
        shape, cdt = ((nb, h, B, d) if kt == "e4m3" else binding.fp4_cache_shape(nb, h, B, d)), torch.uint8
    fill = lambda: torch.full(shape, 3, dtype=cdt, device="cuda")
    want = [fill(), fill()]
    qo, ko = binding.pkv_qk_norm_rope(q, k, cs, pos, *w, interleaved=inter)
    binding.pkv_reshape_and_cache(ko, v.contiguous(), *want, slots, kv_scale=kv)
    got = [fill(), fill()]
    q2 = binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, *got, slots, *w, interleaved=inter, kv_scale=kv)
    assert binding.pkv_get_device_status() == 0
    assert torch.equal(q2, qo)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_positions_and_slots_are_flagged_and_skipped():
    T, hq, h, d, B, nb = 6, 4, 2, 128, 16, 2
    q, k, v, w, cs, pos = make(T, hq, h, d, 128, "bf16", "bf16", max_pos=50)
    good = binding.pkv_qk_norm_rope(q, k, cs, pos, *w)
    bad = pos.clone()
    bad[1], bad[4] = 50, -1
    qo, ko = torch.full_like(good[0], 5.0), torch.full_like(good[1], 5.0)
    binding.pkv_qk_norm_rope(q, k, cs, bad, *w, q_out=qo, k_out=ko)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_POSITION
    for t in range(T):
        for o, g in ((qo, good[0]), (ko, good[1])):
            assert torch.equal(o[t], g[t]) if t not in (1, 4) else (o[t] == 5).all()
    # with the cache: a bad position writes nothing, a bad or negative slot only the query
    kc, vc = (torch.full((nb, h, B, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([3, 4, -1, nb * B, 5, 20], device="cuda")
    qo.fill_(5.0)
    binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, bad, kc, vc, slots, *w, q_out=qo)
    assert binding.pkv_get_device_status() == binding.DEV_BAD_POSITION | binding.DEV_BAD_SLOT
    wk, wv = torch.full_like(kc, 9.0), torch.full_like(vc, 9.0)
    for t in (0, 5):
        s = int(slots[t])
        wk[s // B, :, s % B], wv[s // B, :, s % B] = good[1][t], v[t]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    for t in range(T):
        assert torch.equal(qo[t], good[0][t]) if t not in (1, 4) else (qo[t] == 5).all()


def test_zero_rows_nan_and_infinite_values_stay_in_their_rows():
    T, hq, h, d, B = 4, 2, 1, 64, 8
    q, k, v, w, cs, pos = make(T, hq, h, d, 64, "f16", "f32")
    ref = binding.pkv_qk_norm_rope(q, k, cs, pos, *w)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[1, 0] = 0
    q2[2, 1, 5] = float("nan")
    v2[0, 0, 3] = float("inf")
    kc, vc = (torch.zeros(2, h, B, d, dtype=torch.float16, device="cuda") for _ in range(2))
    slots = torch.arange(T, device="cuda")
    qo = binding.pkv_qk_norm_rope_and_cache(q2, k2, v2, cs, pos, kc, vc, slots, *w)
    assert (qo[1, 0] == 0).all() and torch.isnan(qo[2, 1]).all()
    keep = torch.ones(T, hq, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(qo[keep], ref[0][keep])
    assert torch.equal(vc[0, :, :T].transpose(0, 1), v2) and torch.equal(kc[0, :, :T].transpose(0, 1), ref[1])


def test_another_stream_and_a_captured_step():
    T, hq, h, d, B = 9, 8, 2, 128, 16
    q, k, v, w, cs, pos = make(T, hq, h, d, 128, "bf16", "bf16")
    kc, vc = (torch.zeros(binding.fp4_cache_shape(3, h, B, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(T, device="cuda") + 7
    ref = binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, kc, vc, slots, *w)
    rk, rv = kc.clone(), vc.clone()
    out = torch.zeros_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kc.zero_(), vc.zero_()
    s.wait_stream(torch.cuda.current_stream())
    binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, kc, vc, slots, *w, q_out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(kc, rk) and torch.equal(vc, rv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, kc, vc, slots, *w, q_out=out)
    out.zero_(), kc.zero_(), vc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(kc, rk) and torch.equal(vc, rv)


def test_outputs_are_ordinary_tensors():
    """Outputs that a call allocates: contiguous, apart from each other, of any mode, and gone when dropped."""
    q = torch.randn(5, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(5, 2, 64, device="cuda", dtype=torch.bfloat16)
    cs = torch.randn(9, 32, device="cuda")
    pos = torch.arange(5, device="cuda")
    qo, ko = binding.pkv_qk_norm_rope(q, k, cs, pos)
    assert qo.shape == q.shape and ko.shape == k.shape and qo.is_contiguous() and ko.is_contiguous()
    assert qo.device == q.device and qo.dtype == q.dtype and not qo.requires_grad
    keep = qo.clone()
    ko.fill_(7)
    assert torch.equal(qo, keep) and (ko == 7).all() and ko._version == 1 and qo._version == 0
    loss = (qo.float().requires_grad_() * 2).sum()
    loss.backward()
    again = ko.resize_(3, 2, 64).reshape(-1).tolist()
    assert again == [7.0] * 384 and torch.equal(qo, keep)
    with torch.inference_mode():
        a, b = binding.pkv_qk_norm_rope(q, k, cs, pos)
        assert a.is_inference() and b.is_inference() and torch.equal(a, qo)
    assert not qo.is_inference() and not ko.is_inference()
    e, f = binding.pkv_qk_norm_rope(q[:0], k[:0], cs, pos[:0])
    assert e.shape == (0, 4, 64) and f.shape == (0, 2, 64)
    torch.cuda.synchronize()
    del qo, ko, a, b, e, f, keep, loss
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        binding.pkv_qk_norm_rope(q, k, cs, pos)
    assert torch.cuda.memory_allocated() == before
