"""The binding's checks of element types: two tensors that a call would read as one type have it."""
import pytest
import torch

from paged_kv_cache_87_gb300 import binding, build

F32, F16, BF16, E4M3, U8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.uint8
T, HQ, H, D, B, NB = 3, 4, 2, 64, 16, 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def z(*shape, dt=F32, dev="cpu"):
    return torch.zeros(*shape, dtype=dt, device=dev)


def write(kt, vt, ct, wt, dev="cpu", four=False):
    shape = binding.fp4_cache_shape(NB, H, B, D) if four else (NB, H, B, D)
    args = (z(T, H, D, dt=kt, dev=dev), z(T, H, D, dt=vt, dev=dev), z(*shape, dt=ct, dev=dev), z(*shape, dt=wt, dev=dev))
    binding.pkv_reshape_and_cache(*args, torch.arange(T, device=dev))
    return args


@pytest.mark.parametrize("kt,vt,ct,wt,four", [
    (F16, BF16, U8, U8, False), (F16, BF16, E4M3, U8, False), (BF16, F16, U8, U8, True),
    (F32, F16, U8, U8, False), (BF16, BF16, BF16, F16, False), (F16, BF16, F16, F16, False),
    (F16, F16, F16, U8, False), (F16, F16, U8, torch.float8_e5m2, False)])
def test_a_write_takes_one_type_of_rows_and_of_caches(kt, vt, ct, wt, four):
    with pytest.raises(ValueError, match="element type"):
        write(kt, vt, ct, wt, four=four)


def decode_args(qt, kt, vt, d, dev="cpu"):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)
    return (z(T, HQ, d, dt=qt, dev=dev), z(NB, H, B, d, dt=kt, dev=dev), z(NB, H, B, d, dt=vt, dev=dev),
            i32(T, 2), i32(T))


@pytest.mark.parametrize("qt,kt,vt", [(BF16, BF16, F16), (F16, F16, BF16), (F32, E4M3, torch.float8_e5m2),
                                      (F32, F32, torch.int32), (BF16, U8, torch.int8)])
def test_attention_takes_caches_of_one_type(qt, kt, vt):
    args = decode_args(qt, kt, vt, 128)
    starts = torch.zeros(T + 1, dtype=torch.int32)
    calls = [lambda: binding.pkv_paged_decode_attention(*args, 32, 0.1),
             lambda: binding.pkv_paged_decode_attention(*args, 32, 0.1, prefix=True),
             lambda: binding.prepare_paged_decode_attention(*args, 32, 0.1),
             lambda: binding.pkv_paged_decode_attention_noalloc(*args, 32, 0.1),
             lambda: binding.pkv_paged_multi_query_attention(*args, starts, 32, 0.1),
             lambda: binding.pkv_paged_tree_attention(*args, starts, torch.zeros(T, dtype=torch.int64), 32, 0.1)]
    for i, call in enumerate(calls):
        if i == 5:      # (the mask is looked at first)
            with pytest.raises(ValueError):
                call()
            continue
        with pytest.raises(ValueError, match="element type"):
            call()


@pytest.mark.gpu
def test_rows_that_are_copied_may_have_each_its_caches_type():
    for kt, vt, ct, wt in ((F16, BF16, F16, BF16), (BF16, torch.int16, BF16, torch.int16), (F32, F32, F32, F32)):
        key, value, k, v = write(kt, vt, ct, wt, dev="cuda")
        key.copy_(torch.randint(-9, 9, key.shape)), value.copy_(torch.randint(-9, 9, key.shape))
        binding.pkv_reshape_and_cache(key, value, k, v, torch.arange(T, device="cuda"))
        assert torch.equal(k[0, :, :T].transpose(0, 1), key) and torch.equal(v[0, :, :T].transpose(0, 1), value)
    write(F16, F16, E4M3, U8, dev="cuda")
    assert binding.pkv_get_device_status() == 0


@pytest.mark.gpu
def test_fp8_caches_come_as_either_type():
    q = torch.randn(T, HQ, 128, device="cuda").half()
    k, v = (torch.randn(NB, H, B, 128, device="cuda").to(E4M3) for _ in range(2))
    _, _, _, table, lens = decode_args(F16, E4M3, E4M3, 128, dev="cuda")
    lens.fill_(20), table[:, 1].fill_(3)
    ref = binding.pkv_paged_decode_attention(q, k, v, table, lens, 32, 0.1)
    for a, b in ((k, v.view(U8)), (k.view(U8), v), (k.view(U8), v.view(U8))):
        assert torch.equal(binding.pkv_paged_decode_attention(q, a, b, table, lens, 32, 0.1), ref)
        assert torch.equal(binding.pkv_paged_decode_attention_noalloc(q, a, b, table, lens, 32, 0.1), ref)
    assert binding.pkv_get_device_status() == 0


def test_a_v_cache_that_is_smaller_or_of_another_shape_is_refused():
    rows, slots = z(T, H, D), torch.arange(T)
    k = z(NB, H, B, D)
    for v in (k[:4], z(NB, H, 2 * B, D), z(NB, 2 * H, B, D), z(NB * H, B, D), z(NB, H, B, 2 * D)):
        with pytest.raises(ValueError, match="v_cache"):
            binding.pkv_reshape_and_cache(rows, rows, k, v, slots)


@pytest.mark.gpu
def test_calls_that_were_always_taken_are_taken():
    """An output given as bytes or integers, larger or not; a v_cache with more blocks than the
    k_cache holds."""
    g = torch.Generator("cuda").manual_seed(0)
    q = torch.randn(T, HQ, 128, generator=g, device="cuda").bfloat16()
    key, value = (torch.randn(4 * B, H, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = z(4, H, B, 128, dt=BF16, dev="cuda"), z(9, H, B, 128, dt=BF16, dev="cuda")
    same = z(4, H, B, 128, dt=BF16, dev="cuda")
    slots = torch.arange(4 * B, device="cuda")
    binding.pkv_reshape_and_cache(key, value, k, v, slots)
    binding.pkv_reshape_and_cache(key, value, k, same, slots)
    assert torch.equal(v[:4], same) and not v[4:].any()
    binding.prepare_reshape_and_cache(key, value, k, v, slots)()
    assert torch.equal(v[:4], same)
    table = torch.arange(4, dtype=torch.int32, device="cuda").expand(T, 4).contiguous()
    lens = torch.tensor([64, 1, 33], dtype=torch.int32, device="cuda")
    args = (q, k, same, table, lens, 64, 0.1)
    ref = binding.pkv_paged_decode_attention(*args)
    for dt, n in ((U8, 2 * q.numel()), (U8, 2 * q.numel() + 64), (torch.int16, q.numel()), (torch.int64, q.numel() // 4)):
        out = z(n, dt=dt, dev="cuda")
        assert binding.pkv_paged_decode_attention(*args, out=out) is out
        assert torch.equal(out.view(U8)[:2 * q.numel()], ref.view(U8).flatten())
        assert not out.view(U8)[2 * q.numel():].any()
    for out in (z(2 * q.numel() - 1, dt=U8, dev="cuda"), z(q.numel(), dt=F16, dev="cuda"), z(q.numel(), dev="cuda")):
        with pytest.raises(ValueError, match="out must have"):
            binding.pkv_paged_decode_attention(*args, out=out)
    assert binding.pkv_get_device_status() == 0
