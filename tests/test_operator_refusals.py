"""Arguments that the norm-and-rotation append and the page operations refuse on
the host, before any CUDA call: no GPU needed."""
import ctypes

import pytest
import torch

from continuous_batching_ragged_gb300 import api, native

P = 0x10000                          # an aligned address that no refused call reads


def cache(**kw):
    f = dict(k=P, v=P, num_blocks=16, block_size=16, num_heads=8, head_dim=128, dtype=native.CB_DTYPE_BF16)
    f.update(kw)
    return native.cb_kv_cache(*(f[n] for n, _ in native.cb_kv_cache._fields_))


def rope(lib, c=None, heads=32, pos=P, slots=P, tokens=4, q_out=P, **kw):
    f = dict(q=P, k=P, v=P, q_stride=32 * 128, k_stride=8 * 128, v_stride=8 * 128, q_weight=P, k_weight=P, cos_sin=P,
             max_positions=100, rot_dim=128, interleaved=0, eps=1e-6)
    f.update(kw)
    a = native.cb_norm_rope(*(f[n] for n, _ in native.cb_norm_rope._fields_))
    return lib.cb_norm_rope_append(ctypes.byref(a), heads, pos, slots, None, tokens, ctypes.byref(c or cache()), q_out, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(slots=None), dict(q_out=None), dict(pos=None),
                                dict(cos_sin=None), dict(tokens=-1), dict(heads=0), dict(q=P + 2), dict(q_out=P + 8),
                                dict(q_weight=P + 4), dict(cos_sin=P + 4), dict(q_stride=32 * 128 - 8), dict(k_stride=1024 - 8),
                                dict(v_stride=8 * 128 + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                dict(max_positions=0)])
def test_norm_rope_invalid(native_lib, kw):
    assert rope(native_lib, **kw) == native.CB_ERR_INVALID
    assert b"cb_norm_rope_append" in native_lib.cb_last_error()


@pytest.mark.parametrize("kw,c", [(dict(rot_dim=8), {}), (dict(rot_dim=144), {}), (dict(rot_dim=-16), {}),
                                  (dict(), dict(head_dim=96)), (dict(), dict(head_dim=256, dtype=native.CB_DTYPE_F32)),
                                  (dict(), dict(dtype=7)), (dict(heads=1 << 20), {})])
def test_norm_rope_unsupported(native_lib, kw, c):
    assert rope(native_lib, cache(**c), **kw) == native.CB_ERR_UNSUPPORTED


def test_norm_rope_null_and_empty(native_lib):
    assert native_lib.cb_norm_rope_append(None, 1, None, None, None, 1, ctypes.byref(cache()), P, None) == native.CB_ERR_INVALID
    assert rope(native_lib, cache(num_blocks=0)) == native.CB_ERR_INVALID
    assert rope(native_lib, tokens=0, q=None) == native.CB_OK


def layers(*caches):
    return (native.cb_kv_cache * len(caches))(*caches)


def fork(lib, ls=None, n=None, tables=P, ctx=P, rows=4, width=4, parents=P, children=P, new=P, forks=2):
    ls = layers(cache(), cache()) if ls is None else ls
    return lib.cb_fork_sequences(ls, len(ls) if n is None else n, tables, ctx, rows, width, parents, children, new, forks, None)


def compact(lib, ls=None, tables=P, ctx=P, seqs=4, width=4, new=P, remap=P, live=P, ws=P, ws_bytes=1 << 20):
    ls = layers(cache(), cache()) if ls is None else ls
    return lib.cb_compact_blocks(ls, len(ls), tables, ctx, seqs, width, new, remap, live, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fork, compact])
@pytest.mark.parametrize("kw", [dict(block_size=32), dict(num_blocks=17), dict(num_heads=4), dict(head_dim=64),
                                dict(dtype=native.CB_DTYPE_F32), dict(k=None), dict(v=None), dict(k=P + 8)])
def test_layers_must_be_alike(native_lib, call, kw):
    assert call(native_lib, layers(cache(), cache(**kw))) == native.CB_ERR_INVALID


@pytest.mark.parametrize("call", [fork, compact])
def test_layer_shapes_refused(native_lib, call):
    assert call(native_lib, layers(cache(num_heads=0))) == native.CB_ERR_INVALID
    assert call(native_lib, layers(cache(head_dim=12))) == native.CB_ERR_UNSUPPORTED
    assert call(native_lib, layers(cache(dtype=9))) == native.CB_ERR_UNSUPPORTED
    assert call(native_lib, layers(cache(num_heads=1 << 20, block_size=1 << 10))) == native.CB_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(n=0), dict(tables=None), dict(ctx=None), dict(parents=None), dict(children=None),
                                dict(new=None), dict(forks=-1), dict(rows=-1), dict(width=-1)])
def test_fork_invalid(native_lib, kw):
    assert fork(native_lib, **kw) == native.CB_ERR_INVALID


def test_fork_count(native_lib):
    """Every fork is checked against all others: their number is bounded."""
    assert fork(native_lib, rows=1 << 18, forks=(1 << 16) + 1) == native.CB_ERR_UNSUPPORTED
    assert fork(native_lib, rows=1 << 18, forks=(1 << 31) - 1) == native.CB_ERR_UNSUPPORTED
    assert b"forks" in native_lib.cb_last_error()


def test_fork_nothing(native_lib):
    assert fork(native_lib, forks=0, tables=None) == native.CB_OK


@pytest.mark.parametrize("kw", [dict(tables=None), dict(ctx=None), dict(new=None), dict(remap=None), dict(live=None), dict(ws=None),
                                dict(ws_bytes=64), dict(ws=P + 16), dict(seqs=-1), dict(width=-1)])
def test_compact_invalid(native_lib, kw):
    assert compact(native_lib, **kw) == native.CB_ERR_INVALID


def test_compact_sizes(native_lib):
    assert compact(native_lib, layers(cache(num_blocks=(1 << 20) + 1)), ws_bytes=1 << 30) == native.CB_ERR_UNSUPPORTED
    assert native_lib.cb_compact_workspace_size(0) == 0
    # header, bitmap and its running counts (one word per 32 pages), holes and movers (half the pool each)
    assert native_lib.cb_compact_workspace_size(10240) == 256 + 2 * 1280 + 2 * 20736


def prefix(lib, c=None, q=P, heads=32, cu=P, ctx=P, tables=P, groups=P, lens=P, num_groups=2, seqs=8, tokens=8, width=64, max_q=1,
           max_ctx=512, scale=0.1, out=P, ws=P, ws_bytes=1 << 40):
    return lib.cb_shared_prefix_attention(q, heads, ctypes.byref(c or cache()), cu, ctx, tables, groups, lens, num_groups, seqs, tokens,
                                          width, max_q, max_ctx, scale, out, ws, ws_bytes, None)


# None of these gets as far as resolving the device's error word, which needs a GPU.
@pytest.mark.parametrize("kw", [dict(q=None), dict(cu=None), dict(ctx=None), dict(tables=None), dict(out=None), dict(heads=0),
                                dict(heads=12), dict(seqs=-1), dict(seqs=0), dict(tokens=0), dict(tokens=4), dict(max_q=0),
                                dict(max_q=9), dict(max_ctx=0), dict(width=10), dict(scale=0.0), dict(scale=float("nan")),
                                dict(q=P + 8), dict(out=P + 8)])
def test_shared_prefix_invalid(native_lib, kw):
    assert prefix(native_lib, **kw) == native.CB_ERR_INVALID
    assert b"cb_shared_prefix_attention" in native_lib.cb_last_error()


@pytest.mark.parametrize("c", [dict(head_dim=64), dict(dtype=native.CB_DTYPE_F32), dict(block_size=8), dict(block_size=48)])
def test_shared_prefix_unsupported(native_lib, c):
    assert prefix(native_lib, cache(**c)) == native.CB_ERR_UNSUPPORTED


def test_shared_prefix_groups_and_workspace(native_lib):
    assert prefix(native_lib, groups=None) == native.CB_ERR_INVALID
    assert prefix(native_lib, lens=None) == native.CB_ERR_INVALID
    assert prefix(native_lib, num_groups=0) == native.CB_ERR_INVALID
    assert prefix(native_lib, num_groups=-1) == native.CB_ERR_INVALID
    assert prefix(native_lib, cache(num_heads=1), heads=129) == native.CB_ERR_UNSUPPORTED
    assert prefix(native_lib, seqs=0, tokens=0) == native.CB_OK
    size = native_lib.cb_shared_prefix_workspace_size
    assert size(ctypes.byref(cache(num_heads=1)), 129, 8, 8, 1, 512) == 0
    assert size(ctypes.byref(cache()), 12, 8, 8, 1, 512) == 0 and size(None, 8, 8, 8, 1, 512) == 0
    n = size(ctypes.byref(cache()), 32, 8, 8, 2, 512)
    assert n > native_lib.cb_attention_workspace_size_gqa(ctypes.byref(cache()), 32, 8, 8, 512)
    assert prefix(native_lib, ws=None) == prefix(native_lib, ws_bytes=n - 1) == prefix(native_lib, ws=P + 16) == native.CB_ERR_INVALID


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


# The binding's own checks come before it asks for CUDA tensors, so host tensors show them.
@pytest.mark.parametrize("shape", [(2, 8, 64), (2, 8, 256), (2, 8, 127), (2, 1024), (2, 8, 128, 1)])
def test_shared_prefix_query_shape(shape):
    """The kernels take rows of the cache's head_dim: q and out of shorter ones would be read and written past their ends."""
    q, cache = bf16(*shape), api.KVCache(bf16(4, 8, 16, 128), bf16(4, 8, 16, 128))
    with pytest.raises(ValueError, match="head_dim"):
        api.cb_shared_prefix_attention(q, cache, i32(0, 1, 2), i32(1, 1), i32(0, 1).view(2, 1), i32(0, 2), i32(0), max_q_len=1,
                                       max_context_len=16, scale=0.1, out=torch.empty_like(q), workspace=None)


@pytest.mark.parametrize("dims", [i32(3), i32(), torch.zeros(4, dtype=torch.int64)])
def test_norm_rope_dims(dims):
    """The kernel reads dims[1]: a shorter tensor is refused, as another type is."""
    q, cache = bf16(2, 8, 128), api.KVCache(bf16(4, 8, 16, 128), bf16(4, 8, 16, 128))
    with pytest.raises(ValueError, match="dims"):
        api.cb_norm_rope_append(q, q, q, torch.zeros(2, dtype=torch.int64), cache, q_out=q, dims=dims)
