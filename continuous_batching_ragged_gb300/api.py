"""Thin Python binding of the C ABI: argument marshalling only.

Functions carry the C names.  Tensors are torch tensors on the current CUDA
device (torch supplies device memory and streams, nothing else); every step
of the computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Sequence

import numpy as np
import torch

from . import native
from .native import check

_DTYPES = {torch.bfloat16: native.CB_DTYPE_BF16, torch.float32: native.CB_DTYPE_F32}


_cuda_ready = False


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    # torch.cuda.current_stream().cuda_stream without building a Stream object (0.2 against 2.9 us a call)
    global _cuda_ready
    if not _cuda_ready:
        torch.cuda.init()
        _cuda_ready = True
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


@dataclasses.dataclass
class KVCache:
    """One layer's paged cache: k, v are [num_blocks, H, block_size, A] tensors."""
    k: torch.Tensor
    v: torch.Tensor

    def __post_init__(self):
        if self.k.shape != self.v.shape or self.k.dim() != 4 or self.k.dtype != self.v.dtype:
            raise ValueError("k and v must be equal-shaped [num_blocks, H, B, A] tensors")
        if self.k.dtype not in _DTYPES:
            raise ValueError(f"unsupported cache dtype {self.k.dtype}")

    @classmethod
    def empty(cls, num_blocks: int, num_heads: int, block_size: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda") -> "KVCache":
        shape = (num_blocks, num_heads, block_size, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device))

    @property
    def num_blocks(self) -> int:
        return self.k.shape[0]

    @property
    def num_heads(self) -> int:
        return self.k.shape[1]

    @property
    def block_size(self) -> int:
        return self.k.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]

    def c_struct(self) -> native.cb_kv_cache:
        num_blocks, num_heads, block_size, head_dim = self.k.shape
        return native.cb_kv_cache(_ptr(self.k), _ptr(self.v), num_blocks, block_size, num_heads, head_dim,
                                  _DTYPES[self.k.dtype])


@dataclasses.dataclass
class QuantKVCache:
    """One layer's paged cache in 8 bits: k, v are [num_blocks, H, block_size, A]
    tensors of float8_e4m3fn, k_scale and v_scale fp32 [num_blocks, H]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        if self.k.shape != self.v.shape or self.k.dim() != 4 or not self.k.dtype == self.v.dtype == torch.float8_e4m3fn:
            raise ValueError("k and v must be equal-shaped [num_blocks, H, B, A] tensors of float8_e4m3fn")
        if not self.k_scale.shape == self.v_scale.shape == self.k.shape[:2]:
            raise ValueError("k_scale and v_scale must be [num_blocks, H]")
        if not self.k_scale.dtype == self.v_scale.dtype == torch.float32:
            raise ValueError("k_scale and v_scale must be fp32")

    @classmethod
    def empty(cls, num_blocks: int, num_heads: int, block_size: int, head_dim: int, device="cuda") -> "QuantKVCache":
        k, v = (torch.empty((num_blocks, num_heads, block_size, head_dim), dtype=torch.float8_e4m3fn, device=device)
                for _ in range(2))
        ks, vs = (torch.empty((num_blocks, num_heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    @property
    def num_blocks(self) -> int:
        return self.k.shape[0]

    @property
    def num_heads(self) -> int:
        return self.k.shape[1]

    @property
    def block_size(self) -> int:
        return self.k.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]

    def c_struct(self) -> native.cb_kv_cache_q8:
        num_blocks, num_heads, block_size, head_dim = self.k.shape
        return native.cb_kv_cache_q8(_ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale), num_blocks,
                                     block_size, num_heads, head_dim)


class KVCacheStack:
    """The caches of a model's layers, all of one shape: the `layers` argument of the
    page operations.  Holds the tensors that the caches have when it is made, and the C
    array that describes them; a cache that gets other tensors needs a new stack."""

    def __init__(self, caches: Sequence[KVCache]):
        self.caches = tuple(KVCache(c.k, c.v) for c in caches)
        if not self.caches:
            raise ValueError("at least one layer")
        self.c_array = (native.cb_kv_cache * len(self.caches))(*(c.c_struct() for c in self.caches))

    def __len__(self) -> int:
        return len(self.caches)


def cb_append_kv(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                 cache: KVCache, stream=None) -> None:
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    c = cache.c_struct()
    check(native.lib().cb_append_kv(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), k_new.shape[0],
                                    ctypes.byref(c), _stream_handle(stream)), "cb_append_kv")


def _token_rows(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype, of: str = "the cache's dtype"):
    """Pointer and token stride of [T, heads, A] rows whose tokens may be strided
    (parts of one projection)."""
    if t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of {of}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    token, head, one = t.stride()
    if (one != 1 and shape[2] > 1) or (head != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.data_ptr(), token if shape[0] > 1 else shape[1] * shape[2]


def cb_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                        cache: KVCache, *, q_out: torch.Tensor, positions: Optional[torch.Tensor] = None,
                        cos_sin: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                        dims: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """cb_norm_rope_append: per-head RMS norm of q and k (where a weight is given),
    the position rotation (where cos_sin, [max_positions, rot_dim] fp32, is given)
    and the append of k and v.  q, k, v: [T, heads, A], tokens may be strided.  With
    `dims`, T is the capacity and dims[1] the step's token count."""
    if q.dim() != 3:
        raise ValueError("q must be [num_tokens, heads, head_dim]")
    if dims is not None and (dims.dtype != torch.int32 or dims.numel() < 2):
        raise ValueError("dims must be int32 [num_seqs, num_tokens, ...]")
    T, heads, _ = q.shape
    c = cache.c_struct()
    dtype, A = cache.k.dtype, c.head_dim
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    if positions is not None and (positions.dtype != torch.int32 or positions.numel() != T):
        raise ValueError("positions must be int32 [num_tokens]")
    max_positions = rot_dim = 0
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be fp32 [max_positions, rot_dim]")
        max_positions, rot_dim = cos_sin.shape
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != dtype or w.numel() != A):
            raise ValueError(f"{name} must be [head_dim] of the cache's dtype")
    q_ptr, q_stride = _token_rows(q, "q", (T, heads, A), dtype)
    k_ptr, k_stride = _token_rows(k, "k", (T, c.num_heads, A), dtype)
    v_ptr, v_stride = _token_rows(v, "v", (T, c.num_heads, A), dtype)
    if q_out.shape != q.shape or q_out.dtype != dtype:
        raise ValueError("q_out must have q's shape and dtype")
    a = native.cb_norm_rope(q_ptr, k_ptr, v_ptr, q_stride, k_stride, v_stride, _ptr(q_weight), _ptr(k_weight),
                            _ptr(cos_sin), max_positions, rot_dim, int(interleaved), eps)
    check(native.lib().cb_norm_rope_append(a, heads, _ptr(positions), _ptr(slot_mapping), _ptr(dims), T, c, _ptr(q_out),
                                           _stream_handle(stream)), "cb_norm_rope_append")
    return q_out


def cb_append_kv_q8(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor, cache: QuantKVCache, *,
                    dims: Optional[torch.Tensor] = None, stream=None) -> None:
    """cb_append_kv_q8: cb_append_kv into a cache in 8 bits.  k_new, v_new: [T, H, A]
    bf16 or fp32, tokens may be strided.  With `dims`, T is the capacity and dims[1]
    the step's token count."""
    if dims is not None and (dims.dtype != torch.int32 or dims.numel() < 2):
        raise ValueError("dims must be int32 [num_seqs, num_tokens, ...]")
    T = slot_mapping.numel()
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    if k_new.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {k_new.dtype}")
    c = cache.c_struct()
    shape = (T, c.num_heads, c.head_dim)
    k_ptr, k_stride = _token_rows(k_new, "k_new", shape, k_new.dtype, "bf16 or fp32")
    v_ptr, v_stride = _token_rows(v_new, "v_new", shape, k_new.dtype, "k_new's dtype")
    check(native.lib().cb_append_kv_q8(k_ptr, v_ptr, _DTYPES[k_new.dtype], k_stride, v_stride, _ptr(slot_mapping),
                                       _ptr(dims), T, c, _stream_handle(stream)), "cb_append_kv_q8")


def cb_gather_kv_q8(cache: QuantKVCache, block_tables: torch.Tensor, cu_keys: torch.Tensor, *,
                    k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor], starts: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """cb_gather_kv_q8: sequence s's cached tokens from starts[s] (0 where not given) on
    to rows cu_keys[s] .. cu_keys[s+1]-1 of k_out and v_out, [rows, H, A] bf16 or fp32
    (either may be None)."""
    if not block_tables.dtype is cu_keys.dtype is torch.int32 or (starts is not None and starts.dtype is not torch.int32):
        raise ValueError("block_tables, cu_keys and starts must be int32")
    S = cu_keys.numel() - 1
    if block_tables.dim() != 2 or block_tables.shape[0] != S or (starts is not None and starts.numel() != S):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq], cu_keys [num_seqs + 1], starts [num_seqs]")
    c = cache.c_struct()
    out = v_out if k_out is None else k_out
    if out is None:
        return
    shape, dtype = out.shape, _DTYPES.get(out.dtype)
    if dtype is None or out.dim() != 3 or shape[1] != c.num_heads or shape[2] != c.head_dim or \
            (v_out is not None and out is not v_out and (v_out.dtype is not out.dtype or v_out.shape != shape)):
        raise ValueError("k_out and v_out must be [rows, H, A] of one dtype, bf16 or fp32")
    check(native.lib().cb_gather_kv_q8(c, _ptr(block_tables), _ptr(cu_keys), _ptr(starts), S, block_tables.shape[1],
                                       shape[0], dtype, _ptr(k_out), _ptr(v_out), _stream_handle(stream)), "cb_gather_kv_q8")


def _stack(layers) -> KVCacheStack:
    return layers if isinstance(layers, KVCacheStack) else KVCacheStack(layers)


def cb_fork_sequences(layers, block_tables: torch.Tensor, context_lens: torch.Tensor, parents: torch.Tensor,
                      children: torch.Tensor, new_blocks: torch.Tensor, stream=None) -> None:
    """cb_fork_sequences: rows `children` of block_tables and context_lens continue
    rows `parents` (full pages shared, a last partial page copied to new_blocks).
    layers: a KVCacheStack, or the layers' caches."""
    for name, t in (("block_tables", block_tables), ("context_lens", context_lens), ("parents", parents),
                    ("children", children), ("new_blocks", new_blocks)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if block_tables.dim() != 2 or context_lens.numel() != block_tables.shape[0]:
        raise ValueError("block_tables must be [rows, max_blocks_per_seq] and context_lens [rows]")
    n = parents.numel()
    if children.numel() != n or new_blocks.numel() != n:
        raise ValueError("parents, children and new_blocks must have one entry per fork")
    ls = _stack(layers)
    check(native.lib().cb_fork_sequences(ls.c_array, len(ls), _ptr(block_tables), _ptr(context_lens),
                                         block_tables.shape[0], block_tables.shape[1], _ptr(parents), _ptr(children),
                                         _ptr(new_blocks), n, _stream_handle(stream)), "cb_fork_sequences")


def cb_compact_workspace_size(num_blocks: int) -> int:
    return int(native.lib().cb_compact_workspace_size(num_blocks))


def cb_compact_blocks(layers, block_tables: torch.Tensor, context_lens: torch.Tensor, *,
                      new_block_tables: torch.Tensor, remap: torch.Tensor, num_live: torch.Tensor,
                      workspace: torch.Tensor, stream=None) -> None:
    """cb_compact_blocks: move the live pages to the lowest ids; new_block_tables (may
    be block_tables), remap [num_blocks] and num_live [1] are written.  layers: a
    KVCacheStack, or the layers' caches."""
    for name, t in (("block_tables", block_tables), ("context_lens", context_lens),
                    ("new_block_tables", new_block_tables), ("remap", remap), ("num_live", num_live)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if block_tables.dim() != 2 or context_lens.numel() != block_tables.shape[0]:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] and context_lens [num_seqs]")
    ls = _stack(layers)
    if new_block_tables.shape != block_tables.shape or remap.numel() != ls.caches[0].num_blocks or num_live.numel() < 1:
        raise ValueError("new_block_tables must be as block_tables, remap [num_blocks], num_live [1]")
    check(native.lib().cb_compact_blocks(
        ls.c_array, len(ls), _ptr(block_tables), _ptr(context_lens), block_tables.shape[0], block_tables.shape[1],
        _ptr(new_block_tables), _ptr(remap), _ptr(num_live), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_handle(stream)), "cb_compact_blocks")


def cb_attention_workspace_size(cache: KVCache, num_seqs: int, num_tokens: int,
                                max_context_len: int) -> int:
    c = cache.c_struct()
    return int(native.lib().cb_attention_workspace_size(ctypes.byref(c), num_seqs, num_tokens,
                                                        max_context_len))


def cb_ragged_attention(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                        context_lens: torch.Tensor, block_tables: torch.Tensor, *,
                        max_q_len: int, max_context_len: int, scale: float, out: torch.Tensor,
                        workspace: Optional[torch.Tensor], stream=None) -> torch.Tensor:
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("context_lens", context_lens),
                    ("block_tables", block_tables)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    c = cache.c_struct()
    ws_ptr = _ptr(workspace) if workspace is not None and workspace.numel() else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(native.lib().cb_ragged_attention(
        _ptr(q), ctypes.byref(c), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables),
        context_lens.shape[0], q.shape[0], block_tables.shape[1], max_q_len, max_context_len,
        float(scale), _ptr(out), ws_ptr, ws_bytes, _stream_handle(stream)), "cb_ragged_attention")
    return out


def cb_padded_attention(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                        context_lens: torch.Tensor, block_tables: torch.Tensor, pad_lens: torch.Tensor, *,
                        max_q_len: int, max_context_len: int, scale: float, out: torch.Tensor,
                        workspace: Optional[torch.Tensor], stream=None) -> torch.Tensor:
    """cb_padded_attention: a left-padded batch; the first pad_lens[s] rows of
    sequence s are padding (masked keys, rows not written)."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("context_lens", context_lens),
                    ("block_tables", block_tables), ("pad_lens", pad_lens)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    c = cache.c_struct()
    ws_ptr = _ptr(workspace) if workspace is not None and workspace.numel() else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(native.lib().cb_padded_attention(
        _ptr(q), ctypes.byref(c), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables), _ptr(pad_lens),
        context_lens.shape[0], q.shape[0], block_tables.shape[1], max_q_len, max_context_len,
        float(scale), _ptr(out), ws_ptr, ws_bytes, _stream_handle(stream)), "cb_padded_attention")
    return out


def cb_attention_workspace_size_gqa(cache: KVCache, num_q_heads: int, num_seqs: int, num_tokens: int,
                                    max_context_len: int) -> int:
    c = cache.c_struct()
    return int(native.lib().cb_attention_workspace_size_gqa(ctypes.byref(c), num_q_heads, num_seqs, num_tokens,
                                                            max_context_len))


def cb_ragged_attention_gqa(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                            context_lens: torch.Tensor, block_tables: torch.Tensor, *,
                            max_q_len: int, max_context_len: int, scale: float, out: torch.Tensor,
                            workspace: Optional[torch.Tensor], stream=None) -> torch.Tensor:
    """cb_ragged_attention with q's heads (q.shape[1]) a multiple of the cache's."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("context_lens", context_lens),
                    ("block_tables", block_tables)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    c = cache.c_struct()
    ws_ptr = _ptr(workspace) if workspace is not None and workspace.numel() else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(native.lib().cb_ragged_attention_gqa(
        _ptr(q), q.shape[1], ctypes.byref(c), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables),
        context_lens.shape[0], q.shape[0], block_tables.shape[1], max_q_len, max_context_len,
        float(scale), _ptr(out), ws_ptr, ws_bytes, _stream_handle(stream)), "cb_ragged_attention_gqa")
    return out


def cb_shared_prefix_workspace_size(cache: KVCache, num_q_heads: int, num_seqs: int, num_tokens: int,
                                    num_groups: int, max_context_len: int) -> int:
    c = cache.c_struct()
    return int(native.lib().cb_shared_prefix_workspace_size(ctypes.byref(c), num_q_heads, num_seqs, num_tokens,
                                                            num_groups, max_context_len))


def cb_shared_prefix_attention(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                               context_lens: torch.Tensor, block_tables: torch.Tensor, cu_groups: torch.Tensor,
                               prefix_lens: torch.Tensor, *, max_q_len: int, max_context_len: int, scale: float,
                               out: torch.Tensor, workspace: Optional[torch.Tensor], stream=None) -> torch.Tensor:
    """cb_shared_prefix_attention: cb_ragged_attention_gqa where the sequences
    cu_groups[g] .. cu_groups[g+1]-1 have their first prefix_lens[g] keys in common."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("context_lens", context_lens), ("block_tables", block_tables),
                    ("cu_groups", cu_groups), ("prefix_lens", prefix_lens)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [num_tokens, heads, head_dim] of the cache's head_dim")
    (S,), (num_groups,), (T, heads, _) = context_lens.shape, prefix_lens.shape, q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != S or cu_seqlens_q.shape[0] != S + 1:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] and cu_seqlens_q [num_seqs + 1]")
    if cu_groups.shape[0] != num_groups + 1:
        raise ValueError("cu_groups must be [num_groups + 1]")
    if out.shape != q.shape or out.dtype != q.dtype or q.dtype != cache.k.dtype:
        raise ValueError("q and out must have one shape and the cache's dtype")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None and workspace.numel():
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    check(native.lib().cb_shared_prefix_attention(
        _ptr(q), heads, cache.c_struct(), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables), _ptr(cu_groups),
        _ptr(prefix_lens), num_groups, S, T, block_tables.shape[1], max_q_len, max_context_len, scale, _ptr(out), ws_ptr,
        ws_bytes, _stream_handle(stream)), "cb_shared_prefix_attention")
    return out


def cb_ragged_attention_q8_workspace_size(cache: QuantKVCache, num_q_heads: int, num_seqs: int, num_tokens: int,
                                          max_context_len: int, num_groups: int = 0) -> int:
    c = cache.c_struct()
    return int(native.lib().cb_ragged_attention_q8_workspace_size(ctypes.byref(c), num_q_heads, num_seqs, num_tokens,
                                                                  num_groups, max_context_len))


def cb_ragged_attention_q8(q: torch.Tensor, cache: QuantKVCache, cu_seqlens_q: torch.Tensor,
                           context_lens: torch.Tensor, block_tables: torch.Tensor, *, max_q_len: int,
                           max_context_len: int, scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor],
                           cu_groups: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """cb_ragged_attention_q8: attention over a cache in 8 bits; q, out [T, heads, A]
    bf16.  With cu_groups and prefix_lens, as in cb_shared_prefix_attention."""
    if not cu_seqlens_q.dtype is context_lens.dtype is block_tables.dtype is torch.int32:
        raise ValueError("cu_seqlens_q, context_lens and block_tables must be int32")
    c = cache.c_struct()
    shape = q.shape
    if len(shape) != 3 or shape[2] != c.head_dim:
        raise ValueError("q must be [num_tokens, heads, head_dim] of the cache's head_dim")
    T, heads, _ = shape
    S = context_lens.numel()
    if context_lens.dim() != 1 or block_tables.dim() != 2 or block_tables.shape[0] != S or cu_seqlens_q.numel() != S + 1:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq], context_lens [num_seqs] and cu_seqlens_q [num_seqs + 1]")
    num_groups = 0
    if cu_groups is not None or prefix_lens is not None:
        if cu_groups is None or prefix_lens is None or cu_groups.numel() != prefix_lens.numel() + 1:
            raise ValueError("cu_groups must be [num_groups + 1], and prefix_lens [num_groups] given with it")
        if not cu_groups.dtype is prefix_lens.dtype is torch.int32:
            raise ValueError("cu_groups and prefix_lens must be int32")
        num_groups = prefix_lens.numel()
    if out.shape != shape or not out.dtype is q.dtype is torch.bfloat16:
        raise ValueError("q and out must have one shape and be bf16")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.nbytes
        if ws_bytes:
            ws_ptr = _ptr(workspace)
    check(native.lib().cb_ragged_attention_q8(
        _ptr(q), heads, c, _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables), _ptr(cu_groups), _ptr(prefix_lens),
        num_groups, S, T, block_tables.shape[1], max_q_len, max_context_len, scale, _ptr(out), ws_ptr, ws_bytes,
        _stream_handle(stream)), "cb_ragged_attention_q8")
    return out


def cb_append_kv_dims(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                      dims: torch.Tensor, cache: KVCache, stream=None) -> None:
    """cb_append_kv with the token count in dims[1] (device); k_new's rows bound it."""
    if slot_mapping.dtype != torch.int64 or dims.dtype != torch.int32:
        raise ValueError("slot_mapping must be int64 and dims int32")
    c = cache.c_struct()
    check(native.lib().cb_append_kv_dims(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(dims),
                                         k_new.shape[0], ctypes.byref(c), _stream_handle(stream)),
          "cb_append_kv_dims")


def cb_plan_step(cache: KVCache, cu_seqlens_q: torch.Tensor, context_lens: torch.Tensor, *,
                 num_tokens: int, max_blocks_per_seq: int, max_q_len: int, max_context_len: int,
                 workspace: torch.Tensor, dims: Optional[torch.Tensor] = None,
                 num_q_heads: Optional[int] = None, stream=None) -> None:
    """Build the step's work lists in `workspace` (sizes are capacities when dims is given).
    num_q_heads: query heads of the planned calls when they differ from the
    cache's (grouped-query attention, cb_plan_step_gqa)."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("context_lens", context_lens)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    c = cache.c_struct()
    rest = (_ptr(cu_seqlens_q), _ptr(context_lens), _ptr(dims), context_lens.shape[0], num_tokens,
            max_blocks_per_seq, max_q_len, max_context_len, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if num_q_heads is None:
        check(native.lib().cb_plan_step(ctypes.byref(c), *rest), "cb_plan_step")
    else:
        check(native.lib().cb_plan_step_gqa(ctypes.byref(c), num_q_heads, *rest), "cb_plan_step_gqa")


def cb_ragged_attention_planned(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                                context_lens: torch.Tensor, block_tables: torch.Tensor, *,
                                max_q_len: int, max_context_len: int, scale: float, out: torch.Tensor,
                                workspace: torch.Tensor, dims: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """cb_ragged_attention over the plan cb_plan_step built in `workspace`.  When
    q has more heads than the cache (grouped-query attention) the call goes to
    cb_ragged_attention_planned_gqa, over a plan made with the same num_q_heads."""
    c = cache.c_struct()
    rest = (ctypes.byref(c), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables), _ptr(dims),
            context_lens.shape[0], q.shape[0], block_tables.shape[1], max_q_len, max_context_len, float(scale),
            _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if q.shape[1] == cache.num_heads:
        check(native.lib().cb_ragged_attention_planned(_ptr(q), *rest), "cb_ragged_attention_planned")
    else:
        check(native.lib().cb_ragged_attention_planned_gqa(_ptr(q), q.shape[1], *rest),
              "cb_ragged_attention_planned_gqa")
    return out


def cb_decode_attention_noalloc(q: torch.Tensor, cache: KVCache, cu_seqlens_q: torch.Tensor,
                                context_lens: torch.Tensor, block_tables: torch.Tensor, *,
                                max_context_len: int, scale: float, out: torch.Tensor,
                                stream=None) -> torch.Tensor:
    """Decode-only attention whose scratch is a fixed array the library reserves
    in device memory, for callers that cannot allocate or lend a workspace."""
    c = cache.c_struct()
    check(native.lib().cb_decode_attention_noalloc(
        _ptr(q), ctypes.byref(c), _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables),
        context_lens.shape[0], q.shape[0], block_tables.shape[1], max_context_len, float(scale),
        _ptr(out), _stream_handle(stream)), "cb_decode_attention_noalloc")
    return out


def cb_check_device_errors(stream=None) -> None:
    check(native.lib().cb_check_device_errors(_stream_handle(stream)), "cb_check_device_errors")


def cb_synth_tokens(out: torch.Tensor, seed: int, kind: int, layer: int, seq_ids: torch.Tensor,
                    positions: torch.Tensor, stream=None) -> torch.Tensor:
    n, H, A = out.shape
    check(native.lib().cb_synth_tokens(_ptr(out), _DTYPES[out.dtype], seed, kind, layer,
                                       _ptr(seq_ids), _ptr(positions), n, H, A,
                                       _stream_handle(stream)), "cb_synth_tokens")
    return out


def cb_synth_fill_cache(pool: torch.Tensor, seed: int, kind: int, layer: int, seq_ids: torch.Tensor,
                        prefix_lens: torch.Tensor, block_tables: torch.Tensor, max_prefix: int,
                        stream=None) -> None:
    NB, H, B, A = pool.shape
    check(native.lib().cb_synth_fill_cache(
        _ptr(pool), _DTYPES[pool.dtype], seed, kind, layer, _ptr(seq_ids), _ptr(prefix_lens),
        _ptr(block_tables), block_tables.shape[0], block_tables.shape[1], NB, B, H, A, max_prefix,
        _stream_handle(stream)), "cb_synth_fill_cache")


# ---------------------------------------------------------------------------
# Host scheduler
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class Batch:
    """Copy of one cb_batch (numpy arrays)."""
    num_decode: int
    max_q_len: int
    max_context_len: int
    cu_seqlens_q: np.ndarray
    context_lens: np.ndarray
    block_tables: np.ndarray
    slot_mapping: np.ndarray
    request_ids: np.ndarray
    evicted_ids: np.ndarray
    preempted_ids: np.ndarray

    @property
    def num_seqs(self) -> int:
        return len(self.context_lens)

    @property
    def T(self) -> int:
        return int(self.cu_seqlens_q[-1])

    @property
    def q_lens(self) -> np.ndarray:
        return np.diff(self.cu_seqlens_q)


def _arr(ptr, n, dtype):
    if n == 0:
        return np.zeros(0, dtype=dtype)
    return np.ctypeslib.as_array(ptr, shape=(n,)).astype(dtype, copy=True)


class Scheduler:
    """cb_scheduler_* on the host (no GPU needed)."""

    def __init__(self, token_budget: int, block_size: int, num_blocks: int, max_num_seqs: int = 0,
                 admission: str = "reserve_lifetime"):
        self._L = native.lib()
        cfg = native.cb_sched_config(token_budget, block_size, num_blocks, max_num_seqs,
                                     native.ADMISSION[admission])
        h = ctypes.c_void_p()
        check(self._L.cb_scheduler_create(ctypes.byref(cfg), ctypes.byref(h)), "cb_scheduler_create")
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._L.cb_scheduler_destroy(h)
            self._h = None

    def add_request(self, rid: int, arrival_step: int, prompt_len: int, output_len: int) -> None:
        check(self._L.cb_add_request(self._h, rid, arrival_step, prompt_len, output_len), "cb_add_request")

    def build_batch(self) -> Batch:
        b = native.cb_batch()
        check(self._L.cb_build_batch(self._h, ctypes.byref(b)), "cb_build_batch")
        S, T, W = b.num_seqs, b.num_tokens, b.max_blocks_per_seq
        return Batch(num_decode=b.num_decode, max_q_len=b.max_q_len, max_context_len=b.max_context_len,
                     cu_seqlens_q=_arr(b.cu_seqlens_q, S + 1, np.int32),
                     context_lens=_arr(b.context_lens, S, np.int32),
                     block_tables=_arr(b.block_tables, S * W, np.int32).reshape(S, W),
                     slot_mapping=_arr(b.slot_mapping, T, np.int64),
                     request_ids=_arr(b.request_ids, S, np.int64),
                     evicted_ids=_arr(b.evicted_ids, b.num_evicted, np.int64),
                     preempted_ids=_arr(b.preempted_ids, b.num_preempted, np.int64))

    def complete_step(self) -> None:
        check(self._L.cb_complete_step(self._h), "cb_complete_step")

    def stats(self) -> native.cb_sched_stats:
        s = native.cb_sched_stats()
        check(self._L.cb_scheduler_stats(self._h, ctypes.byref(s)), "cb_scheduler_stats")
        return s

    @property
    def idle(self) -> bool:
        s = self.stats()
        return s.num_waiting == 0 and s.num_running == 0
