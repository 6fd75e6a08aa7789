"""Serving operators of ``libgdn.so`` (see include/gdn.h, "serving"): the binding.

One step of a stack that interleaves gated-delta layers with attention layers: ``paged_plan``
turns request lengths into block tables, slots and offsets on the GPU, ``paged_write`` puts
the step's keys and values into the pages, ``paged_attention`` attends over them, and
``recurrent_step`` carries the gated delta rule over the step's tokens on a pool of states.
Argument checks and marshalling only; every call is asynchronous on the given (default: the
current) stream.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from .gdn import _check, _dtype_code, load_library


class PagedPlan(NamedTuple):
    """What ``paged_plan`` returns: int32 tensors on the requests' device."""
    cu_seqlens: torch.Tensor   # [N + 1] offsets of the requests' new tokens
    seq_lens: torch.Tensor     # [N] tokens held after the step
    slot_map: torch.Tensor     # [T] cache slot of each new token, -1: none
    positions: torch.Tensor    # [T] position of each new token
    granted: torch.Tensor      # [N] 1: the request got its blocks
    ring_state: torch.Tensor   # [2] for the next call


_same_device = contextlib.nullcontext()


def _on(dev: torch.device):
    """The library works on the current device, which must be the tensors' device."""
    return _same_device if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(stream: Optional[torch.cuda.Stream], dev: torch.device) -> int:
    return (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream


def _fail(fn: str, name: str, t, want: str):
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"
    raise ValueError(f"{fn}: {name} must be {want}, got {got}")


def _need(fn: str, name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, dev) -> int:
    """A contiguous CUDA tensor of this dtype, shape and device; its address."""
    if (t is None or t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_cuda or
            not t.is_contiguous()):
        _fail(fn, name, t, f"a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def _rows(fn: str, name: str, t: torch.Tensor, dtype: torch.dtype, dev) -> int:
    """[T, heads, d] with dense heads and any token stride; the token stride in elements."""
    if (t.dim() != 3 or t.dtype != dtype or t.device != dev or not t.is_cuda or
            t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        _fail(fn, name, t, f"a {dtype} CUDA tensor [T, heads, d] on {dev} with dense heads")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def gdn_paged_plan(context_lens, new_lens, block_tables, free_ring, ring_in, ring_out, cu_seqlens,
                   seq_lens, slot_map, positions, granted, block_size: int,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name: contiguous int32 CUDA
    tensors, the last six of them outputs."""
    fn, i32, dev = "gdn_paged_plan", torch.int32, context_lens.device
    N, T, nb = context_lens.numel(), slot_map.numel(), free_ring.numel()
    if block_tables.dim() != 2:
        _fail(fn, "block_tables", block_tables, "[N, max_blocks]")
    M = block_tables.shape[1]
    ptrs = [_need(fn, name, t, i32, shape, dev) for name, t, shape in (
        ("context_lens", context_lens, (N,)), ("new_lens", new_lens, (N,)),
        ("block_tables", block_tables, (N, M)), ("free_ring", free_ring, (nb,)),
        ("ring_in", ring_in, (2,)), ("ring_out", ring_out, (2,)),
        ("cu_seqlens", cu_seqlens, (N + 1,)), ("seq_lens", seq_lens, (N,)),
        ("slot_map", slot_map, (T,)), ("positions", positions, (T,)), ("granted", granted, (N,)))]
    with _on(dev):
        _check(load_library().gdn_paged_plan(*ptrs, N, T, M, nb, block_size, _stream(stream, dev)))


def paged_plan(context_lens, new_lens, block_tables, free_ring, ring_state, block_size: int,
               num_tokens: int) -> PagedPlan:
    """Block tables, slots and offsets of one step.  context_lens, new_lens [N] (new_lens
    below 0: the request has ended); block_tables [N, max_blocks] and free_ring
    [num_blocks] are updated in place; ring_state [2] (first free entry, free entries);
    num_tokens is the room for new tokens (their sum, or more).  All int32 on the GPU; the
    next call takes the returned ring_state."""
    N = context_lens.numel()
    buf = torch.empty(3 * N + 3 + 2 * num_tokens, dtype=torch.int32, device=context_lens.device)
    cu, seq, granted, ring, slots, pos = buf.split((N + 1, N, N, 2, num_tokens, num_tokens))
    gdn_paged_plan(context_lens, new_lens, block_tables, free_ring, ring_state, ring, cu, seq, slots,
                   pos, granted, block_size)
    return PagedPlan(cu, seq, slots, pos, granted, ring)


def gdn_paged_write(k, v, slot_map, k_cache, v_cache,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name: k, v [T, Hkv, d] (any token
    stride that is a multiple of 16 bytes) into k_cache, v_cache [num_blocks, block_size,
    Hkv, d] at slot_map [T] int32."""
    fn, dev, dt = "gdn_paged_write", k_cache.device, k_cache.dtype
    code = _dtype_code(dt)
    if k_cache.dim() != 4:
        _fail(fn, "k_cache", k_cache, "[num_blocks, block_size, Hkv, d]")
    nb, bs, H, d = k_cache.shape
    ks, vs, T = _rows(fn, "k", k, dt, dev), _rows(fn, "v", v, dt, dev), k.shape[0]
    if k.shape[1:] != (H, d) or v.shape != k.shape:
        raise ValueError(f"{fn}: k and v must be [T, {H}, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    slots = _need(fn, "slot_map", slot_map, torch.int32, (T,), dev)
    kc = _need(fn, "k_cache", k_cache, dt, k_cache.shape, dev)
    vc = _need(fn, "v_cache", v_cache, dt, k_cache.shape, dev)
    with _on(dev):
        _check(load_library().gdn_paged_write(k.data_ptr(), v.data_ptr(), slots, kc, vc, T, H, d, nb,
                                              bs, ks, vs, code, _stream(stream, dev)))


def paged_write(k, v, slot_map, k_cache, v_cache) -> None:
    """Write the step's keys and values into the pages, on the current stream."""
    gdn_paged_write(k, v, slot_map, k_cache, v_cache)


def gdn_paged_attention_workspace_bytes(heads: int, kv_heads: int, d: int, max_q_len: int,
                                        dtype: torch.dtype) -> int:
    """Device workspace ``gdn_paged_attention`` needs on the current device."""
    return int(load_library().gdn_paged_attention_workspace_bytes(heads, kv_heads, d, max_q_len,
                                                                  _dtype_code(dtype)))


def gdn_paged_attention(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
                        max_q_len: int, max_seq_len: int = 0, scale: Optional[float] = None,
                        window: int = 0, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name.  q [T, Hq, d] (any token
    stride that is a multiple of 16 bytes), out [T, Hq, d], lse [T, Hq] fp32 or None; the
    caches as for ``gdn_paged_write``; block_tables [N, max_blocks], seq_lens [N] and
    cu_seqlens [N + 1] int32; workspace a CUDA uint8 tensor; scale None: d ** -0.5."""
    fn, dev, dt = "gdn_paged_attention", q.device, q.dtype
    code = _dtype_code(dt)
    qs = _rows(fn, "q", q, dt, dev)
    if k_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError(f"{fn}: k_cache must be [num_blocks, block_size, Hkv, d] and block_tables "
                         f"[N, max_blocks], got {tuple(k_cache.shape)} and {tuple(block_tables.shape)}")
    T, Hq, d = q.shape
    nb, bs, Hkv, dc = k_cache.shape
    N, M = block_tables.shape
    if dc != d:
        raise ValueError(f"{fn}: q and k_cache have different head sizes ({d}, {dc})")
    i32 = torch.int32
    kc = _need(fn, "k_cache", k_cache, dt, k_cache.shape, dev)
    vc = _need(fn, "v_cache", v_cache, dt, k_cache.shape, dev)
    bt = _need(fn, "block_tables", block_tables, i32, (N, M), dev)
    sl = _need(fn, "seq_lens", seq_lens, i32, (N,), dev)
    cu = _need(fn, "cu_seqlens", cu_seqlens, i32, (N + 1,), dev)
    op = _need(fn, "out", out, dt, q.shape, dev)
    lp = None if lse is None else _need(fn, "lse", lse, torch.float32, (T, Hq), dev)
    if not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        _fail(fn, "workspace", workspace, f"a contiguous CUDA tensor on {dev}")
    with _on(dev):
        _check(load_library().gdn_paged_attention(
            q.data_ptr(), kc, vc, bt, sl, cu, op, lp, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), N, T, Hq, Hkv, d, M, nb, bs, max_q_len,
            max_seq_len, window, d ** -0.5 if scale is None else scale, qs, code, _stream(stream, dev)))


def paged_attention(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, max_q_len: int,
                    max_seq_len: int = 0, scale: Optional[float] = None, window: int = 0,
                    return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of each request's new tokens over its pages (causal; with ``window`` > 0
    the last ``window`` tokens only).  Returns out [T, Hq, d], and lse [T, Hq] fp32 with
    ``return_lse``.  max_q_len: the most new tokens of a request; max_seq_len: the most
    tokens of a sequence if known; ``workspace`` to bring one's own scratch."""
    T, Hq, d = q.shape
    out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        if k_cache.dim() != 4:
            _fail("paged_attention", "k_cache", k_cache, "[num_blocks, block_size, Hkv, d]")
        with _on(q.device):
            nbytes = gdn_paged_attention_workspace_bytes(Hq, k_cache.shape[2], d, max_q_len, q.dtype)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    gdn_paged_attention(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
                        max_q_len, max_seq_len, scale, window)
    return (out, lse) if return_lse else out


def gdn_recurrent_step(q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out,
                       context_lens=None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name.  q, k [T, Hk, dk] and
    v [T, H, dv] (any token stride that is a multiple of 16 bytes); log_alpha, beta [T, H]
    fp32; state_pool [slots, H, dv, dk] fp32, updated in place; state_index [N],
    cu_seqlens [N + 1] and context_lens [N] or None int32; out [T, H, dv]."""
    fn, dev, dt = "gdn_recurrent_step", v.device, v.dtype
    code = _dtype_code(dt)
    qs, ks, vs = (_rows(fn, name, t, dt, dev) for name, t in (("q", q), ("k", k), ("v", v)))
    T, Hk, dk = k.shape
    H, dv = v.shape[1:]
    if q.shape != k.shape or v.shape[0] != T or state_pool.dim() != 4:
        raise ValueError(f"{fn}: need q, k [T, Hk, dk], v [T, H, dv] and state_pool [slots, H, dv, dk], "
                         f"got {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}, {tuple(state_pool.shape)}")
    f32, i32, N, slots = torch.float32, torch.int32, state_index.numel(), state_pool.shape[0]
    la = _need(fn, "log_alpha", log_alpha, f32, (T, H), dev)
    be = _need(fn, "beta", beta, f32, (T, H), dev)
    sp = _need(fn, "state_pool", state_pool, f32, (slots, H, dv, dk), dev)
    si = _need(fn, "state_index", state_index, i32, (N,), dev)
    cu = _need(fn, "cu_seqlens", cu_seqlens, i32, (N + 1,), dev)
    cl = None if context_lens is None else _need(fn, "context_lens", context_lens, i32, (N,), dev)
    op = _need(fn, "out", out, dt, (T, H, dv), dev)
    with _on(dev):
        _check(load_library().gdn_recurrent_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), la, be, sp, si, cu, cl, op, N, T, Hk, H, dk, dv,
            slots, qs, ks, vs, code, _stream(stream, dev)))


def recurrent_step(q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens,
                   context_lens=None) -> torch.Tensor:
    """The gated delta rule over each request's new tokens on the pool of states (updated in
    place), on the current stream.  Returns out [T, H, dv]."""
    out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    gdn_recurrent_step(q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out, context_lens)
    return out
