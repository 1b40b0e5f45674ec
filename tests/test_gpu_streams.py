"""Calls that take memory for another stream than the current one: it is neither memory that the
current stream's queued work still uses, nor given out again while that stream reads the result."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding

pytestmark = pytest.mark.gpu

CALLS = ["decode", "gather", "norm", "norm and write", "multi-query", "draft trees", "without a workspace"]
BUSY = 40_000_000          # cycles: some 20 ms


def step():
    """Inputs of every call that allocates, long ready on the device, and the calls by name: each
    takes a stream and gives a list of its outputs."""
    g = torch.Generator("cuda").manual_seed(1)
    T, hq, h, d, B, nb = 512, 8, 2, 128, 16, 40
    kc, vc = (torch.zeros(binding.fp4_cache_shape(nb, h, B, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    q, k, v = (torch.randn(T, n, d, generator=g, device="cuda").bfloat16() for n in (hq, h, h))
    slots = torch.randperm(nb * B, generator=g, device="cuda")[:T]
    cs = torch.cat([torch.ones(T, 64), torch.zeros(T, 64)], 1).cuda()
    pos = torch.arange(T, device="cuda")
    binding.pkv_reshape_and_cache(k, v, kc, vc, slots)
    k16, v16 = (torch.randn(nb, h, B, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None].expand(T, nb).contiguous()
    lens = i32([600] * T)
    rows = i32([0, T])
    chain = i32(list(range(0, T + 1, 8)))
    tree = torch.full((T,), 1, dtype=torch.int64, device="cuda")
    calls = {
        "decode": lambda s: [binding.pkv_paged_decode_attention(q, kc, vc, table, lens, 640, 0.1, stream=s)],
        "gather": lambda s: binding.pkv_gather_cache(kc, vc, table[:1], rows, T, torch.bfloat16, stream=s),
        "norm": lambda s: binding.pkv_qk_norm_rope(q, k, cs, pos, stream=s),
        "norm and write": lambda s: [binding.pkv_qk_norm_rope_and_cache(q, k, v, cs, pos, kc, vc, slots, stream=s)],
        "multi-query": lambda s: [binding.pkv_paged_multi_query_attention(
            q, k16, v16, table[:T // 8], lens[:T // 8], chain, 640, 0.1, stream=s)],
        "draft trees": lambda s: [binding.pkv_paged_tree_attention(
            q, k16, v16, table[:T // 8], lens[:T // 8], chain, tree, 640, 0.1, stream=s)],
        "without a workspace": lambda s: [binding.pkv_paged_decode_attention_noalloc(
            q[:32], k16, v16, table[:32], lens[:32], 640, 0.1, stream=s)],
    }
    return calls


def drop_while_read(tensor):
    """Queues a long delay and then a reader of `tensor` on the current stream: what it reads."""
    seen = torch.empty_like(tensor)
    torch.cuda._sleep(BUSY)
    seen.copy_(tensor)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_leaves_what_the_current_one_still_reads(name):
    call = step()[name]
    ref = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = {t.untyped_storage().nbytes() for t in call(None)}
    need = [binding.pkv_decode_workspace_bytes(512, 8, 2, 128, 16, 640, "e2m1"),
            binding.pkv_multi_query_workspace_bytes(64)]
    for size in sorted(sizes) + need:            # a block that would fit the output, or the workspace
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        x = torch.full((size,), 17, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        seen = drop_while_read(x)
        del x
        out = call(side)
        torch.cuda.synchronize()
        assert (seen == 17).all()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("name", CALLS)
def test_an_output_dropped_while_the_current_stream_reads_it_is_not_written_again(name):
    call = step()[name]
    ref = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    seen = [drop_while_read(t) for t in out]
    del out
    trash = []
    with torch.cuda.stream(side):
        for t in ref:
            trash += [torch.full_like(t, 9.0) for _ in range(4)]
    again = call(side)
    torch.cuda.synchronize()
    assert len(trash) == 4 * len(ref)
    assert all(torch.equal(a, b) for a, b in zip(seen, ref))
    assert all(torch.equal(a, b) for a, b in zip(again, ref))
    assert binding.pkv_get_device_status() == 0


def test_block_pairs_from_the_host_outlive_the_call():
    """Pairs that a call stages for itself stay until its stream has read them."""
    nb, h, B, d = 64, 2, 16, 128
    k, v = (torch.randn(nb, h, B, d, device="cuda").half() for _ in range(2))
    pairs = [[i, 32 + i] for i in range(32)]
    other = torch.tensor([[i, 63 - i] for i in range(32)], dtype=torch.int32)
    want = [torch.cat([x[:32], x[:32]]) for x in (k, v)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    binding.pkv_copy_blocks(k, v, pairs, stream=side)
    trash = [other.cuda() for _ in range(16)]
    torch.cuda.synchronize()
    assert len(trash) == 16 and torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("kind", ["list", "array", "tensor"])
def test_swap_pairs_from_the_host_outlive_the_call(kind):
    """The pinned buffer that a swap stages its pairs in, whatever they came as."""
    nb, h, B, d = 64, 2, 16, 128
    k, v = (torch.randn(nb, h, B, d, device="cuda").half() for _ in range(2))
    hk, hv = (torch.zeros(nb, h, B, d, dtype=torch.float16).pin_memory() for _ in range(2))
    pairs = [[i, 63 - i] for i in range(32)]
    other = torch.tensor([[63 - i, i] for i in range(32)], dtype=torch.int32)
    given = {"list": pairs, "array": np.array(pairs), "tensor": torch.tensor(pairs)}[kind]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    binding.pkv_swap_blocks(k, v, hk, hv, given, stream=side)
    trash = [other.clone().pin_memory() for _ in range(16)]
    torch.cuda.synchronize()
    want = torch.zeros(2, nb, h, B, d, dtype=torch.float16)
    for a, b in pairs:
        want[0, b], want[1, b] = k[a].cpu(), v[a].cpu()
    assert len(trash) == 16 and torch.equal(hk, want[0]) and torch.equal(hv, want[1])
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("name", CALLS)
def test_the_default_stream_asked_for_under_another_one(name):
    """The other way round: work is current on a side stream, the call goes to the default one."""
    call = step()[name]
    ref = [t.clone() for t in call(None)]
    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x = [torch.full((t.untyped_storage().nbytes(),), 17, dtype=torch.uint8, device="cuda") for t in ref]
        torch.cuda.synchronize()
        seen = [drop_while_read(t) for t in x]
        del x
        out = call(default)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert all((t == 17).all() for t in seen)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert binding.pkv_get_device_status() == 0


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_a_stream_that_joins_a_capture(name):
    """Captured on a side stream of the graph's own, with memory of the graph's pool; two graphs."""
    call = step()[name]
    ref = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            outs.append(call(side))
            torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, ref))
    assert binding.pkv_get_device_status() == 0
