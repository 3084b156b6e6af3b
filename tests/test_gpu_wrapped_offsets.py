"""Query offsets and context lengths whose difference does not fit 32 bits: the sequence is reported and left out, by every attention call."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TOP, LOW = 2 ** 31 - 1, -2 ** 31


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(kind, H, K, A, q_lens, ctx, width):
    from continuous_batching_ragged_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(5)
    blocks, dt = len(ctx) * width, torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "q8":
        cache = api.QuantKVCache(*(torch.randn((blocks, K, 16, A), generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)),
                                 *(torch.ones((blocks, K), device="cuda") for _ in range(2)))
    else:
        cache = api.KVCache(*(torch.randn((blocks, K, 16, A), generator=g, device="cuda").to(dt) for _ in range(2)))
    T = sum(q_lens)
    q = torch.randn((T, H, A), generator=g, device="cuda").to(dt)
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").view(len(ctx), width)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return cache, q, tables, cu


def call(kind, cache, q, tables, cu, ctx, max_q, max_ctx, out):
    from continuous_batching_ragged_gb300 import api
    S, T, H = ctx.numel(), q.shape[0], q.shape[1]
    kw = dict(max_q_len=max_q, max_context_len=max_ctx, scale=1 / math.sqrt(q.shape[2]), out=out)
    if kind == "noalloc":
        api.cb_decode_attention_noalloc(q, cache, cu, ctx, tables, max_context_len=max_ctx, scale=kw["scale"], out=out)
        return
    if kind in ("bf16", "f32"):
        n, f, args = api.cb_attention_workspace_size(cache, S, T, max_ctx), api.cb_ragged_attention, ()
    elif kind == "gqa":
        n, f, args = api.cb_attention_workspace_size_gqa(cache, H, S, T, max_ctx), api.cb_ragged_attention_gqa, ()
    elif kind == "prefix":
        n, f, args = api.cb_shared_prefix_workspace_size(cache, H, S, T, 1, max_ctx), api.cb_shared_prefix_attention, (ints([0, S]), ints([0]))
    else:
        n, f, args = api.cb_ragged_attention_q8_workspace_size(cache, H, S, T, max_ctx), api.cb_ragged_attention_q8, ()
    f(q, cache, cu, ctx, tables, *args, workspace=torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"), **kw)


# the calls, and the steps that take each of their paths: few sequences, more than a CTA has threads, chunks
CASES = [("noalloc", 4, 4, 1, 6), ("f32", 4, 4, 1, 6), ("f32", 4, 4, 9, 6), ("bf16", 4, 4, 1, 6), ("bf16", 4, 4, 140, 6), ("gqa", 16, 2, 1, 6),
         ("gqa", 16, 2, 140, 6), ("prefix", 8, 2, 1, 6), ("prefix", 8, 2, 1, 600), ("prefix", 8, 2, 140, 6), ("q8", 8, 2, 1, 6),
         ("q8", 8, 2, 1, 600), ("q8", 8, 2, 140, 6)]


@pytest.mark.parametrize("kind,H,K,n,S", CASES)
def test_wrapped_offsets(native_lib, kind, H, K, n, S):
    from continuous_batching_ragged_gb300 import api, native
    ctx = [n + (13 * s) % 60 for s in range(S)]
    cache, q, tables, cu = make(kind, H, K, 128, [n] * S, ctx, -(-(n + 60) // 16))
    good = torch.full_like(q, float("nan"))
    call(kind, cache, q, tables, ints(cu), ints(ctx), n, max(ctx), good)
    api.cb_check_device_errors()
    assert bool(good.isfinite().all())
    bad = cu[:-2] + [TOP - n // 2, LOW + n - 1 - n // 2]  # the last one's offsets are n apart in 32 bits, the one's before it far apart
    out = torch.full_like(q, float("nan"))
    call(kind, cache, q, tables, ints(bad), ints(ctx), n, max(ctx), out)
    with pytest.raises(native.CBError) as e:
        api.cb_check_device_errors()
    assert e.value.status == native.CB_ERR_INVALID
    at = cu[-3]
    assert bool(out[at:].isnan().all())
    # the others' keys may be cut otherwise: both are within half a step of bf16 and of their weights' rounding
    assert bool(((out[:at].float() - good[:at].float()).abs() <= 2 ** -6 * (1 + good[:at].float().abs())).all())


@pytest.mark.parametrize("kind", ["prefix", "q8"])
def test_wrapped_group(native_lib, kind):
    """A group whose first sequence's length and query tokens are 2^31 apart and more shares nothing."""
    from continuous_batching_ragged_gb300 import api, native
    S, p = 600, 2048
    ctx = [p + 1 + s % 30 for s in range(S)]
    cache, q, tables, cu = make("q8" if kind == "q8" else "bf16", 32, 2, 128, [1] * S, ctx, 131)
    tables[:, :p // 16] = tables[0, :p // 16].clone()
    for wrong_ctx, wrong_cu in ((LOW, 1), (-100, LOW + 50)):
        c, u = list(ctx), list(cu)
        c[0], u[1] = wrong_ctx, wrong_cu
        if kind == "q8":
            n, f = api.cb_ragged_attention_q8_workspace_size(cache, 32, S, S, max(ctx), num_groups=1), api.cb_ragged_attention_q8
        else:
            n, f = api.cb_shared_prefix_workspace_size(cache, 32, S, S, 1, max(ctx)), api.cb_shared_prefix_attention
        out = torch.full_like(q, float("nan"))
        f(q, cache, ints(u), ints(c), tables, cu_groups=ints([0, S]), prefix_lens=ints([p]), max_q_len=1, max_context_len=max(ctx),
          scale=1 / math.sqrt(128), out=out, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        with pytest.raises(native.CBError) as e:
            api.cb_check_device_errors()
        assert e.value.status == native.CB_ERR_INVALID
        assert bool(out[0].isnan().all()) and bool(out[2:].isfinite().all())
