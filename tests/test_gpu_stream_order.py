"""Operators that may start while the stream's last kernel ends, behind work of other kinds:
a mixed step whose decode kernel ends long before its prefill kernel, copies, fills, other
streams, eagerly and captured."""
import pytest
import torch

pytestmark = pytest.mark.gpu

A, B, H, K = 128, 16, 16, 8


def bf16(*shape, g):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("prefix", [False, True])
def test_behind_a_mixed_step(native_lib, prefix):
    """One long chunk and one decode row: what comes next overwrites the step's queries and keys."""
    from continuous_batching_ragged_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(3)
    chunk, ctx = 3000, [9000, 40]
    blocks = [-(-c // B) for c in ctx]
    first = api.KVCache(bf16(sum(blocks), K, B, A, g=g), bf16(sum(blocks), K, B, A, g=g))
    tables = torch.full((2, max(blocks)), -1, dtype=torch.int32, device="cuda")
    tables[0, :blocks[0]] = torch.arange(blocks[0], device="cuda")
    tables[1, :blocks[1]] = torch.arange(blocks[0], sum(blocks), device="cuda")
    q = bf16(chunk + 1, H, A, g=g)
    new_q, new_kv = bf16(chunk + 1, H, A, g=g), bf16(chunk + 1, K, A, g=g)
    slots = torch.arange(chunk + 1, device="cuda")
    ws = torch.empty(api.cb_attention_workspace_size_gqa(first, H, 2, chunk + 1, max(ctx)), dtype=torch.uint8, device="cuda")
    cu, lens = i32([0, chunk, chunk + 1]), i32(ctx)

    def step(q, cache, out):
        api.cb_ragged_attention_gqa(q, cache, cu, lens, tables, max_q_len=chunk, max_context_len=max(ctx), scale=A ** -0.5, out=out,
                                    workspace=ws)

    def follow(q, cache, small):
        if prefix:                                     # reads the cache, writes over the step's queries
            api.cb_shared_prefix_attention(new_q[:2], cache, i2, l2, tables, g2, p2, max_q_len=1, max_context_len=max(ctx),
                                           scale=A ** -0.5, out=q[:2], workspace=small)
        else:                                          # writes over its queries and keys
            api.cb_norm_rope_append(new_q, new_kv, new_kv, slots, cache, q_out=q)

    i2, l2, g2, p2 = i32([0, 1, 2]), i32([500, 40]), i32([0, 2]), i32([0])
    small = torch.empty(api.cb_shared_prefix_workspace_size(first, H, 2, 2, 1, max(ctx)), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(q)
    step(q, first, want)
    torch.cuda.synchronize()
    got = torch.empty_like(q)
    for _ in range(3):
        q2, cache = q.clone(), api.KVCache(first.k.clone(), first.v.clone())
        got.fill_(float("nan"))
        step(q2, cache, got)
        follow(q2, cache, small)
        api.cb_check_device_errors()
        assert torch.equal(got, want)
    q2, cache = q.clone(), api.KVCache(first.k.clone(), first.v.clone())
    q3, k3, v3 = q.clone(), first.k.clone(), first.v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2.copy_(q3)
        cache.k.copy_(k3)
        cache.v.copy_(v3)
        step(q2, cache, got)
        follow(q2, cache, small)
    for _ in range(3):
        got.fill_(float("nan"))
        graph.replay()
        api.cb_check_device_errors()
        assert torch.equal(got, want)


@pytest.mark.parametrize("captured", [False, True])
def test_behind_copies_fills_and_another_stream(native_lib, captured):
    from continuous_batching_ragged_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(4)
    T = 600
    cache = api.KVCache(bf16(64, K, B, A, g=g), bf16(64, K, B, A, g=g))
    stack = api.KVCacheStack([cache])
    src, q, kv = bf16(T, H, A, g=g), torch.empty((T, H, A), dtype=torch.bfloat16, device="cuda"), bf16(T, K, A, g=g)
    slots, out = torch.arange(T, device="cuda"), torch.empty_like(q)
    tables, lens = torch.full((4, 64), -1, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    tables0 = tables.clone()
    tables0[0, :38] = torch.arange(38, device="cuda")
    lens0 = i32([T, 0, 0, 0])
    parents, children, new = i32([0, 0]), i32([1, 2]), i32([40, 41])
    att = torch.empty((3, H, A), dtype=torch.bfloat16, device="cuda")
    n = api.cb_shared_prefix_workspace_size(cache, H, 3, 3, 1, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cws = torch.empty(api.cb_compact_workspace_size(64), dtype=torch.uint8, device="cuda")
    remap, live = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    cu, groups, prefix, tables3, lens3 = i32([0, 1, 2, 3]), i32([0, 3]), i32([T - 1]), tables[:3], lens[:3]
    side = torch.cuda.Stream()

    def work():
        here = torch.cuda.current_stream()
        q.copy_(src)                                   # a copy, then two branches that join
        side.wait_stream(here)
        with torch.cuda.stream(side):
            tables.copy_(tables0)
            lens.copy_(lens0)
        cache.k.fill_(0)
        cache.v.fill_(0)
        api.cb_norm_rope_append(q, kv, kv, slots, cache, q_out=out)
        here.wait_stream(side)
        api.cb_fork_sequences(stack, tables, lens, parents, children, new)
        att.fill_(0)
        api.cb_shared_prefix_attention(out[:3], cache, cu, lens3, tables3, groups, prefix, max_q_len=1, max_context_len=T,
                                       scale=A ** -0.5, out=att, workspace=ws)
        api.cb_compact_blocks(stack, tables3, lens3, new_block_tables=tables3, remap=remap, num_live=live, workspace=cws)

    torch.cuda.synchronize()
    run = work
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        run = graph.replay
    for _ in range(5):
        for t in (out, att, q):
            t.fill_(float("nan"))
        run()
        api.cb_check_device_errors()
        assert torch.equal(out, src)
        assert int(live) == 40 and lens.tolist() == [T, T, T, 0] and tables[1, 37] == 38 and tables[2, 37] == 39
        k = cache.k[tables[2, :38].long()].transpose(1, 2).reshape(-1, K, A)[:T]
        assert torch.equal(k, kv)
        s = torch.einsum("shgd,jhd->shgj", src[:3].double().view(3, K, H // K, A), kv.double()) * A ** -0.5
        want = torch.einsum("shgj,jhd->shgd", torch.softmax(s, -1), kv.double()).reshape(3, H, A)
        # P and the output rounded to bf16, 2^-8 each of values below 5; sums of 128 products below 40 in fp32
        assert float((att.double() - want).abs().max()) < 5 * 3 * 2.0 ** -8
