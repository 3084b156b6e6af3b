"""Arguments that the calls on caches in 8 bits refuse on the host, before any CUDA call: no GPU needed."""
import ctypes

import pytest
import torch

from continuous_batching_ragged_gb300 import api, native

P = 0x10000                          # an aligned address that no refused call reads


def cache(**kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, num_blocks=16, block_size=16, num_heads=8, head_dim=128)
    f.update(kw)
    return native.cb_kv_cache_q8(*(f[n] for n, _ in native.cb_kv_cache_q8._fields_))


def append(lib, c=None, k=P, v=P, dtype=native.CB_DTYPE_BF16, k_stride=1024, v_stride=1024, slots=P, tokens=4):
    return lib.cb_append_kv_q8(k, v, dtype, k_stride, v_stride, slots, None, tokens, ctypes.byref(c or cache()), None)


def gather(lib, c=None, tables=P, cu=P, starts=None, seqs=2, width=4, rows=8, dtype=native.CB_DTYPE_BF16, k=P, v=P):
    return lib.cb_gather_kv_q8(ctypes.byref(c or cache()), tables, cu, starts, seqs, width, rows, dtype, k, v, None)


def attend(lib, c=None, q=P, heads=32, cu=P, ctx=P, tables=P, groups=None, lens=None, num_groups=0, seqs=8, tokens=8, width=64, max_q=1,
           max_ctx=512, scale=0.1, out=P, ws=P, ws_bytes=1 << 40):
    return lib.cb_ragged_attention_q8(q, heads, ctypes.byref(c or cache()), cu, ctx, tables, groups, lens, num_groups, seqs, tokens, width,
                                      max_q, max_ctx, scale, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(slots=None), dict(tokens=-1), dict(k=P + 8), dict(v=P + 2),
                                dict(k_stride=1016), dict(v_stride=1023), dict(k_stride=1028),
                                dict(dtype=native.CB_DTYPE_F32, v_stride=1026)])
def test_append_invalid(native_lib, kw):
    assert append(native_lib, **kw) == native.CB_ERR_INVALID
    assert b"cb_append_kv_q8" in native_lib.cb_last_error()


@pytest.mark.parametrize("call", [append, gather])
def test_cache_refused(native_lib, call):
    for kw in (dict(num_blocks=0), dict(block_size=0), dict(num_heads=-1), dict(head_dim=0), dict(k=None), dict(v_scale=None), dict(k=P + 8)):
        assert call(native_lib, cache(**kw)) == native.CB_ERR_INVALID, kw
    for kw in (dict(head_dim=96), dict(block_size=48), dict(block_size=2048), dict(num_heads=1 << 20)):
        assert call(native_lib, cache(**kw)) == native.CB_ERR_UNSUPPORTED, kw


def test_append_sizes(native_lib):
    assert append(native_lib, tokens=0, k=None) == native.CB_OK
    assert append(native_lib, tokens=65537) == native.CB_ERR_UNSUPPORTED
    assert append(native_lib, dtype=7) == native.CB_ERR_UNSUPPORTED
    assert append(native_lib, cache(head_dim=256), dtype=native.CB_DTYPE_F32, k_stride=2048, v_stride=2048) == native.CB_ERR_UNSUPPORTED
    assert append(native_lib, cache(num_heads=65536), tokens=65536, k_stride=1 << 24, v_stride=1 << 24) == native.CB_ERR_UNSUPPORTED
    assert native_lib.cb_append_kv_q8(P, P, 1, 1024, 1024, P, None, 4, None, None) == native.CB_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(tables=None), dict(cu=None), dict(seqs=-1), dict(width=-1), dict(rows=-1), dict(k=P + 8), dict(v=P + 4)])
def test_gather_invalid(native_lib, kw):
    assert gather(native_lib, **kw) == native.CB_ERR_INVALID


def test_gather_nothing(native_lib):
    assert gather(native_lib, rows=0, k=None) == gather(native_lib, seqs=0) == gather(native_lib, k=None, v=None) == native.CB_OK
    assert gather(native_lib, dtype=5) == native.CB_ERR_UNSUPPORTED
    assert native_lib.cb_gather_kv_q8(None, P, P, None, 1, 1, 1, 1, P, P, None) == native.CB_ERR_INVALID


# None of these gets as far as resolving the device's error word, which needs a GPU.
@pytest.mark.parametrize("kw", [dict(q=None), dict(cu=None), dict(ctx=None), dict(tables=None), dict(out=None), dict(heads=0),
                                dict(heads=12), dict(seqs=-1), dict(seqs=0), dict(tokens=0), dict(tokens=4), dict(max_q=0),
                                dict(max_q=9), dict(max_ctx=0), dict(width=10), dict(scale=0.0), dict(scale=float("nan")),
                                dict(q=P + 8), dict(out=P + 8), dict(groups=P), dict(lens=P), dict(num_groups=1), dict(num_groups=-1),
                                dict(groups=P, lens=P), dict(groups=P, num_groups=1), dict(ws=None), dict(ws=P + 16), dict(ws_bytes=100)])
def test_attention_invalid(native_lib, kw):
    assert attend(native_lib, **kw) == native.CB_ERR_INVALID
    assert b"cb_ragged_attention_q8" in native_lib.cb_last_error()


def test_attention_caches(native_lib):
    for kw in (dict(head_dim=64), dict(head_dim=256), dict(block_size=8), dict(block_size=48), dict(block_size=256)):
        assert attend(native_lib, cache(**kw)) == native.CB_ERR_UNSUPPORTED, kw
    for kw in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(v=P + 4), dict(num_blocks=0)):
        assert attend(native_lib, cache(**kw)) == native.CB_ERR_INVALID, kw
    assert attend(native_lib, cache(num_heads=1), heads=129) == native.CB_ERR_UNSUPPORTED
    assert attend(native_lib, seqs=0, tokens=0) == native.CB_OK
    assert native_lib.cb_ragged_attention_q8(P, 8, None, P, P, P, None, None, 0, 1, 1, 64, 1, 16, 0.1, P, P, 1 << 40, None) == native.CB_ERR_INVALID


def test_attention_workspace(native_lib):
    size = native_lib.cb_ragged_attention_q8_workspace_size
    assert size(ctypes.byref(cache(num_heads=1)), 129, 8, 8, 0, 512) == 0
    assert size(ctypes.byref(cache()), 12, 8, 8, 0, 512) == 0 and size(None, 8, 8, 8, 0, 512) == 0
    n = size(ctypes.byref(cache()), 32, 8, 8, 0, 512)
    assert n > 0 and attend(native_lib, ws_bytes=n - 1) == native.CB_ERR_INVALID
    assert b"workspace too small" in native_lib.cb_last_error()
    assert size(ctypes.byref(cache()), 32, 8, 8, 4, 512) >= n


def q8(*shape, **kw):
    t = dict(k=torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn), v=torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn),
             k_scale=torch.ones(shape[:2]), v_scale=torch.ones(shape[:2]))
    t.update(kw)
    return api.QuantKVCache(**t)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("kw", [dict(k=bf16(4, 8, 16, 128)), dict(k_scale=torch.ones(4, 9)), dict(v_scale=torch.ones(4, 8, 1)),
                                dict(k_scale=torch.ones(4, 8, dtype=torch.float64)),
                                dict(v=torch.zeros((4, 8, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn))])
def test_binding_cache(kw):
    with pytest.raises(ValueError):
        q8(4, 8, 16, 128, **kw)


# The binding's own checks come before it asks for CUDA tensors, or are what it says of host tensors.
def test_binding_append():
    c, slots = q8(4, 8, 16, 128), torch.zeros(2, dtype=torch.int64)
    for k, v, s, d in ((bf16(2, 8, 128), bf16(2, 8, 128), slots.int(), None), (bf16(2, 8, 128).half(), bf16(2, 8, 128), slots, None),
                       (bf16(2, 8, 128), bf16(2, 8, 128), slots, i32(2)), (bf16(2, 8, 128), bf16(2, 8, 128), slots, None)):
        with pytest.raises(ValueError):
            api.cb_append_kv_q8(k, v, s, c, dims=d)


def test_binding_gather():
    c = q8(4, 8, 16, 128)
    out = bf16(4, 8, 128)
    for tables, cu, starts, k in ((i32(0).view(1, 1), i32(0, 4), i32(0, 0), out), (i32(0), i32(0, 4), None, out),
                                  (i32(0).view(1, 1), i32(0, 4).long(), None, out), (i32(0).view(1, 1), i32(0, 4), None, out.half()),
                                  (i32(0).view(1, 1), i32(0, 4), None, bf16(4, 8, 64))):
        with pytest.raises(ValueError):
            api.cb_gather_kv_q8(c, tables, cu, k_out=k, v_out=None, starts=starts)
    with pytest.raises(ValueError):
        api.cb_gather_kv_q8(c, i32(0).view(1, 1), i32(0, 4), k_out=out, v_out=bf16(5, 8, 128))


@pytest.mark.parametrize("kw", [dict(q=bf16(2, 8, 64)), dict(q=bf16(2, 1024)), dict(q=torch.zeros(2, 8, 128)), dict(cu=i32(0, 1)),
                                dict(tables=i32(0, 1)), dict(cu_groups=i32(0, 2)), dict(prefix_lens=i32(0)),
                                dict(cu_groups=i32(0, 2), prefix_lens=i32(0, 0)), dict(ctx=i32(1, 1).long())])
def test_binding_attention(kw):
    f = dict(q=bf16(2, 8, 128), cu=i32(0, 1, 2), ctx=i32(1, 1), tables=i32(0, 1).view(2, 1), cu_groups=None, prefix_lens=None)
    f.update(kw)
    with pytest.raises(ValueError):
        api.cb_ragged_attention_q8(f["q"], q8(4, 8, 16, 128), f["cu"], f["ctx"], f["tables"], max_q_len=1, max_context_len=16, scale=0.1,
                                   out=torch.empty_like(f["q"]), workspace=None, cu_groups=f["cu_groups"], prefix_lens=f["prefix_lens"])


def test_workspace_without_groups(native_lib):
    """A step without groups has no room for shared prefixes' records: two a row and 131,072 more."""
    c = cache()

    def size(seqs, tokens, groups, ctx):
        return native_lib.cb_ragged_attention_q8_workspace_size(ctypes.byref(c), 32, seqs, tokens, groups, ctx)

    for seqs, tokens, ctx in ((64, 64, 4096), (67, 2050, 4096), (2000, 2000, 512)):
        assert size(seqs, tokens, 1, ctx) - size(seqs, tokens, 0, ctx) >= 20 << 20
    assert 0 < size(64, 64, 0, 4096) <= 60 << 20
    assert size(1, 1, 0, 64) == size(1, 1, 1, 64)     # the records of the whole grid's shares are more
