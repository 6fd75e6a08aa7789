"""Serving operators of ``libgdn.so`` (see include/gdn.h, "serving"): the binding.

One step of a stack that interleaves gated-delta layers with attention layers: ``paged_plan``
turns request lengths into block tables, slots and offsets on the GPU, ``paged_write`` puts
the step's keys and values into the pages, ``paged_attention`` attends over them, and
``recurrent_step`` carries the gated delta rule over the step's tokens on a pool of states.
Argument checks and marshalling only; every call is asynchronous on the given (default: the
current) stream.

A small step is as long as its host side: the kernels of eight requests take 3 to 10 us.  So
the checks here read a tensor's properties once and build no messages until one fails, and
the calls that allocate their outputs do not check them again (us a call on the host: plan
35 -> 24, attention 35 -> 24, write 14 -> 8, step 24 -> 15).
"""
from __future__ import annotations

import contextlib
import functools
from typing import NamedTuple, Optional

import torch

from .gdn import _check, _dtype_code, load_library

_I32, _F32 = torch.int32, torch.float32


class PagedPlan(NamedTuple):
    """What ``paged_plan`` returns: int32 tensors on the requests' device."""
    cu_seqlens: torch.Tensor   # [N + 1] offsets of the requests' new tokens
    seq_lens: torch.Tensor     # [N] tokens held after the step
    slot_map: torch.Tensor     # [T] cache slot of each new token, -1: none
    positions: torch.Tensor    # [T] position of each new token
    granted: torch.Tensor      # [N] 1: the request got its blocks
    ring_state: torch.Tensor   # [2] for the next call


_same_device = contextlib.nullcontext()


def _on(dev: int):
    """The library works on the current device, which must be the tensors' device."""
    return _same_device if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(stream: Optional[torch.cuda.Stream], dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _fail(fn: str, name: str, t, want: str):
    got = type(t).__name__ if not torch.is_tensor(t) else f"{t.dtype} {tuple(t.shape)} on {t.device}"
    raise ValueError(f"{fn}: {name} must be {want}, got {got}")


def _device(fn: str, name: str, t) -> int:
    """Index of the CUDA device that holds t."""
    dev = t.get_device()
    if dev < 0:
        _fail(fn, name, t, "a CUDA tensor")
    return dev


def _need(fn: str, name: str, t, dtype, shape, dev: int) -> int:
    """A contiguous tensor of this type, shape and device; its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _fail(fn, name, t, f"a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _rows(fn: str, name: str, t, dtype, dev: int) -> int:
    """[T, heads, d] with dense heads and any token stride; the token stride in elements."""
    if t.dtype is not dtype or t.dim() != 3 or t.get_device() != dev:
        _fail(fn, name, t, f"a {dtype} tensor [T, heads, d] on cuda:{dev}")
    (T, H, d), (st, sh, sd) = t.shape, t.stride()
    if (sd != 1 and d > 1) or (sh != d and H > 1):
        _fail(fn, name, t, "[T, heads, d] with dense heads")
    return st if T > 1 else H * d


def gdn_paged_plan(context_lens, new_lens, block_tables, free_ring, ring_in, ring_out, cu_seqlens,
                   seq_lens, slot_map, positions, granted, block_size: int,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name: contiguous int32 CUDA
    tensors, the last six of them outputs."""
    fn = "gdn_paged_plan"
    N, T = context_lens.numel(), slot_map.numel()
    dev = _device(fn, "context_lens", context_lens)
    out = [_need(fn, name, t, _I32, shape, dev) for name, t, shape in (
        ("ring_out", ring_out, (2,)), ("cu_seqlens", cu_seqlens, (N + 1,)), ("seq_lens", seq_lens, (N,)),
        ("slot_map", slot_map, (T,)), ("positions", positions, (T,)), ("granted", granted, (N,)))]
    _plan(fn, dev, context_lens, new_lens, block_tables, free_ring, ring_in, out, T, block_size, stream)


def _plan(fn, dev, context_lens, new_lens, block_tables, free_ring, ring_in, out, T, block_size, stream):
    N, nb = context_lens.numel(), free_ring.numel()
    if block_tables.dim() != 2:
        _fail(fn, "block_tables", block_tables, "[N, max_blocks]")
    M = block_tables.shape[1]
    cl = _need(fn, "context_lens", context_lens, _I32, (N,), dev)
    nl = _need(fn, "new_lens", new_lens, _I32, (N,), dev)
    bt = _need(fn, "block_tables", block_tables, _I32, (N, M), dev)
    fr = _need(fn, "free_ring", free_ring, _I32, (nb,), dev)
    ri = _need(fn, "ring_in", ring_in, _I32, (2,), dev)
    with _on(dev):
        _check(load_library().gdn_paged_plan(cl, nl, bt, fr, ri, *out, N, T, M, nb, block_size,
                                             _stream(stream, dev)))


def paged_plan(context_lens, new_lens, block_tables, free_ring, ring_state, block_size: int,
               num_tokens: int) -> PagedPlan:
    """Block tables, slots and offsets of one step.  context_lens, new_lens [N] (new_lens
    below 0: the request has ended); block_tables [N, max_blocks] and free_ring
    [num_blocks] are updated in place; ring_state [2] (first free entry, free entries);
    num_tokens is the room for new tokens (their sum, or more).  All int32 on the GPU; the
    next call takes the returned ring_state."""
    dev = _device("paged_plan", "context_lens", context_lens)
    N, T = context_lens.numel(), num_tokens
    # one allocation for the six outputs
    buf = torch.empty(3 * N + 3 + 2 * T, dtype=_I32, device=context_lens.device)
    sizes = (N + 1, N, T, T, N, 2)
    cu = buf.data_ptr()
    seq = cu + 4 * (N + 1)
    slots = seq + 4 * N
    pos = slots + 4 * T
    granted = pos + 4 * T
    ring = granted + 4 * N
    if T == 0:  # nothing to point at
        slots = pos = None
    _plan("paged_plan", dev, context_lens, new_lens, block_tables, free_ring, ring_state,
          (ring, cu, seq, slots, pos, granted), T, block_size, None)
    return PagedPlan._make(buf.split_with_sizes(sizes))


def gdn_paged_write(k, v, slot_map, k_cache, v_cache,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name: k, v [T, Hkv, d] (any token
    stride that is a multiple of 16 bytes) into k_cache, v_cache [num_blocks, block_size,
    Hkv, d] at slot_map [T] int32."""
    fn, dt = "gdn_paged_write", k_cache.dtype
    code, dev = _dtype_code(dt), _device(fn, "k_cache", k_cache)
    shape = k_cache.shape
    if len(shape) != 4:
        _fail(fn, "k_cache", k_cache, "[num_blocks, block_size, Hkv, d]")
    nb, bs, H, d = shape
    ks, vs = _rows(fn, "k", k, dt, dev), _rows(fn, "v", v, dt, dev)
    T = k.shape[0]
    if k.shape != (T, H, d) or v.shape != (T, H, d):
        raise ValueError(f"{fn}: k and v must be [T, {H}, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    slots = _need(fn, "slot_map", slot_map, _I32, (T,), dev)
    kc = _need(fn, "k_cache", k_cache, dt, shape, dev)
    vc = _need(fn, "v_cache", v_cache, dt, shape, dev)
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


@functools.lru_cache(maxsize=256)
def _workspace_bytes(dev: int, heads: int, kv_heads: int, d: int, max_q_len: int, dtype) -> int:
    with _on(dev):
        return gdn_paged_attention_workspace_bytes(heads, kv_heads, d, max_q_len, dtype)


def gdn_paged_attention(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
                        max_q_len: int, max_seq_len: int = 0, scale: Optional[float] = None,
                        window: int = 0, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name.  q [T, Hq, d] (any token
    stride that is a multiple of 16 bytes), out [T, Hq, d], lse [T, Hq] fp32 or None; the
    caches as for ``gdn_paged_write``; block_tables [N, max_blocks], seq_lens [N] and
    cu_seqlens [N + 1] int32; workspace a CUDA uint8 tensor; scale None: d ** -0.5."""
    fn = "gdn_paged_attention"
    dev = _device(fn, "q", q)
    _need(fn, "out", out, q.dtype, q.shape, dev)
    if lse is not None:
        _need(fn, "lse", lse, _F32, q.shape[:2], dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _fail(fn, "workspace", workspace, f"a contiguous tensor on cuda:{dev}")
    _attention(fn, dev, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
               max_q_len, max_seq_len, scale, window, stream)


def _attention(fn, dev, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
               max_q_len, max_seq_len, scale, window, stream):
    dt, shape = q.dtype, k_cache.shape
    code = _dtype_code(dt)
    qs = _rows(fn, "q", q, dt, dev)
    T, Hq, d = q.shape
    if len(shape) != 4 or shape[3] != d or block_tables.dim() != 2:
        raise ValueError(f"{fn}: k_cache must be [num_blocks, block_size, Hkv, {d}] and block_tables "
                         f"[N, max_blocks], got {tuple(shape)} and {tuple(block_tables.shape)}")
    nb, bs, Hkv, _ = shape
    N, M = block_tables.shape
    kc = _need(fn, "k_cache", k_cache, dt, shape, dev)
    vc = _need(fn, "v_cache", v_cache, dt, shape, dev)
    bt = _need(fn, "block_tables", block_tables, _I32, (N, M), dev)
    sl = _need(fn, "seq_lens", seq_lens, _I32, (N,), dev)
    cu = _need(fn, "cu_seqlens", cu_seqlens, _I32, (N + 1,), dev)
    with _on(dev):
        _check(load_library().gdn_paged_attention(
            q.data_ptr(), kc, vc, bt, sl, cu, out.data_ptr(), None if lse is None else lse.data_ptr(),
            workspace.data_ptr(), workspace.nbytes, N, T, Hq, Hkv, d, M, nb, bs, max_q_len, max_seq_len,
            window, d ** -0.5 if scale is None else scale, qs, code, _stream(stream, dev)))


def paged_attention(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, max_q_len: int,
                    max_seq_len: int = 0, scale: Optional[float] = None, window: int = 0,
                    return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of each request's new tokens over its pages (causal; with ``window`` > 0
    the last ``window`` tokens only).  Returns out [T, Hq, d], and lse [T, Hq] fp32 with
    ``return_lse``.  max_q_len: the most new tokens of a request; max_seq_len: the most
    tokens of a sequence if known; ``workspace`` to bring one's own scratch."""
    fn = "paged_attention"
    dev, device = _device(fn, "q", q), q.device
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError(f"{fn}: q must be [T, Hq, d] and k_cache [num_blocks, block_size, Hkv, d], got "
                         f"{tuple(q.shape)} and {tuple(k_cache.shape)}")
    T, Hq, d = q.shape
    out = torch.empty((T, Hq, d), dtype=q.dtype, device=device)
    lse = torch.empty((T, Hq), dtype=_F32, device=device) if return_lse else None
    if workspace is None:
        nbytes = _workspace_bytes(dev, Hq, k_cache.shape[2], d, max_q_len, q.dtype)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _fail(fn, "workspace", workspace, f"a contiguous tensor on cuda:{dev}")
    _attention(fn, dev, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, out, lse, workspace,
               max_q_len, max_seq_len, scale, window, None)
    return (out, lse) if return_lse else out


def gdn_recurrent_step(q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out,
                       context_lens=None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Tensor-level call of the C entry point of the same name.  q, k [T, Hk, dk] and
    v [T, H, dv] (any token stride that is a multiple of 16 bytes); log_alpha, beta [T, H]
    fp32; state_pool [slots, H, dv, dk] fp32, updated in place; state_index [N],
    cu_seqlens [N + 1] and context_lens [N] or None int32; out [T, H, dv]."""
    fn = "gdn_recurrent_step"
    dev = _device(fn, "v", v)
    _need(fn, "out", out, v.dtype, v.shape, dev)
    _step(fn, dev, q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out, context_lens, stream)


def _step(fn, dev, q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out, context_lens, stream):
    dt = v.dtype
    code = _dtype_code(dt)
    qs, ks, vs = _rows(fn, "q", q, dt, dev), _rows(fn, "k", k, dt, dev), _rows(fn, "v", v, dt, dev)
    T, Hk, dk = k.shape
    _, H, dv = v.shape
    if q.shape != (T, Hk, dk) or v.shape[0] != T or state_pool.dim() != 4:
        raise ValueError(f"{fn}: need q, k [T, Hk, dk], v [T, H, dv] and state_pool [slots, H, dv, dk], "
                         f"got {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}, {tuple(state_pool.shape)}")
    N, slots = state_index.numel(), state_pool.shape[0]
    la = _need(fn, "log_alpha", log_alpha, _F32, (T, H), dev)
    be = _need(fn, "beta", beta, _F32, (T, H), dev)
    sp = _need(fn, "state_pool", state_pool, _F32, (slots, H, dv, dk), dev)
    si = _need(fn, "state_index", state_index, _I32, (N,), dev)
    cu = _need(fn, "cu_seqlens", cu_seqlens, _I32, (N + 1,), dev)
    cl = None if context_lens is None else _need(fn, "context_lens", context_lens, _I32, (N,), dev)
    with _on(dev):
        _check(load_library().gdn_recurrent_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), la, be, sp, si, cu, cl, out.data_ptr(), N, T, Hk, H,
            dk, dv, slots, qs, ks, vs, code, _stream(stream, dev)))


def recurrent_step(q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens,
                   context_lens=None) -> torch.Tensor:
    """The gated delta rule over each request's new tokens on the pool of states (updated in
    place), on the current stream.  Returns out [T, H, dv]."""
    dev = _device("recurrent_step", "v", v)
    out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _step("recurrent_step", dev, q, k, v, log_alpha, beta, state_pool, state_index, cu_seqlens, out,
          context_lens, None)
    return out
