"""The full-attention layer's operators: residual norm, rotary append to a paged 8-bit cache,
attention over that cache.

The calls of ``include/kda.h``'s section on the full-attention layer, on torch tensors; like
the rest of the binding, marshalling only.  A cache is four tensors and two indexes:

    k_cache, v_cache   float8_e4m3fn (or uint8) [pages, kv_heads, page_size, 128], any strides
                       that are multiples of 16 with the channels dense
    k_scale, v_scale   fp32 [pages, kv_heads]
    block_table        int32 [num_seqs, max_blocks]: the pages of each sequence, in order
    kv_lens            int32 [num_seqs]: cached tokens, the step's new ones included

A call with ``stream`` allocates its outputs and workspace on that stream; the tensors given to it
must be ready there.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import operator
import os
import struct
import warnings

import torch

from . import (ERR_INVALID_ARG, HEAD_DIM, KDAError, OK, STATE_BF16, STATE_F32, _elsewhere,
               _within, lib)

_BF16, _F32 = torch.bfloat16, torch.float32
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_DENSE = torch.contiguous_format
_HALF, _EITHER = (_BF16,), (_BF16, _F32)
_FLOAT = (_F32,)
_I32 = torch.int32
_INT = (_I32,)
_UINT8 = (torch.uint8,)
# the current stream's handle without a Stream object around it (a call's host time counts in decode)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# The usual calls' marshalling in C++ (csrc/kda_layer_binding.cpp): with it a call of 14 rows of the
# norm takes 5.6 us of the host instead of 14.2, an append 7.4 instead of 20.1, attention 8.0 instead
# of 23.1.  It returns None for whatever is not usual, errors included, and the code below then
# takes the call.
_native = None


class _NoneUsual:
    """In the module's place where it was not built, or for another torch: every call is the Python
    code's."""
    add_rms_norm = rope_append = cached_attention = staticmethod(lambda *args: None)


def _load_native():
    global _native
    from .build import binding_path
    path = binding_path()
    if not os.path.exists(path):
        warnings.warn(f"{path} is missing (kda_gated_delta_chunk_gb300.build.build() makes it): small calls of "
                      "the attention layer's operators take some 10 us more of the host", RuntimeWarning, 3)
        _native = _NoneUsual
        return _native
    loader = importlib.machinery.ExtensionFileLoader("_layer", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_layer", path, loader=loader))
    loader.exec_module(module)
    L = lib()
    module.entries(*(ctypes.cast(f, ctypes.c_void_p).value
                     for f in (L.kda_add_rms_norm, L.kda_rope_append, L.kda_cached_attention)))
    _native = module
    return module


# kda_kv_cache of kda.h, as ``_cache`` packs it
_CACHE = struct.Struct("@PPPPqqqqiiiiPqP")


def _check(t, name, dtypes, shape, dev, dense_from=1):
    """Type, device (its index) and shape; dimensions from ``dense_from`` on are dense.  Returns the stride of
    the first dimension.  (Kept short for the usual contiguous tensor: a decode step's calls are
    bound by their host time.)"""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in dtypes
            and t.shape == shape and t.is_contiguous()):
        return t.stride(0) if shape[0] != 1 else t.numel()
    return _check_slowly(t, name, dtypes, shape, dev, dense_from)


def _check_slowly(t, name, dtypes, shape, dev, dense_from):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    inner = 1
    sizes, strides = t.shape, t.stride()
    for d in range(len(sizes) - 1, dense_from - 1, -1):
        if strides[d] != inner and sizes[d] > 1:
            raise ValueError(f"{name}: only the first {dense_from} dimension(s) may be strided"
                             if dense_from else f"{name} must be contiguous")
        inner *= sizes[d]
    # a dimension of one element takes the dense stride: torch leaves it arbitrary
    return strides[0] if sizes[0] > 1 else t.numel()


def _need_cuda(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _i32(x, name):
    """A number the entry points take in 32 bits (ctypes would cut a larger one to them)."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise KDAError(ERR_INVALID_ARG, f"{name} {x} does not fit 32 bits")
    return x


def _stream(stream, dev):
    return stream.cuda_stream if stream is not None else _raw_stream(dev)


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, num_seqs, dev):
    """The packed kda_kv_cache, and its number of kv heads."""
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, 128]")
    pages, hk, page, d = shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    blocks = block_table.size(-1) if block_table.dim() == 2 else -1
    scales = (pages, hk)
    # the usual case at once: everything contiguous, of the right type, shape and device
    if (k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous() and block_table.is_contiguous() and kv_lens.is_contiguous()
            and k_cache.dtype in _BYTES and v_cache.dtype in _BYTES and k_scale.dtype is _F32
            and v_scale.dtype is _F32 and block_table.dtype is _I32 and kv_lens.dtype is _I32
            and v_cache.shape == shape and k_scale.shape == scales and v_scale.shape == scales
            and block_table.shape == (num_seqs, blocks) and kv_lens.shape == (num_seqs,)
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and k_scale.get_device() == dev and v_scale.get_device() == dev
            and block_table.get_device() == dev and kv_lens.get_device() == dev):
        tok, row, sc = HEAD_DIM, blocks, hk
        head = page * HEAD_DIM
        per_page = hk * head
    else:
        per_page = _check(k_cache, "k_cache", _BYTES, shape, dev, 3)
        _check(v_cache, "v_cache", _BYTES, shape, dev, 3)
        st = k_cache.stride()
        if v_cache.stride() != st:
            raise ValueError("k_cache and v_cache must have the same strides")
        sc = _check(k_scale, "k_scale", _FLOAT, scales, dev)
        if _check(v_scale, "v_scale", _FLOAT, scales, dev) != sc:
            raise ValueError("k_scale and v_scale must have the same strides")
        if blocks < 0:
            raise ValueError("block_table must be [num_seqs, max_blocks]")
        row = _check(block_table, "block_table", _INT, (num_seqs, blocks), dev)
        _check(kv_lens, "kv_lens", _INT, (num_seqs,), dev, 0)
        tok = st[2] if page > 1 else HEAD_DIM
        head = st[1] if hk > 1 else page * tok
        if pages == 1:
            per_page = hk * head
        if num_seqs == 1:
            row = blocks
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                       per_page, head, tok, sc, pages, page, hk, blocks, block_table.data_ptr(), row,
                       kv_lens.data_ptr()), hk


def _status_workspace(workspace, dev):
    if workspace is None:
        return torch.zeros(256, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", _UINT8, workspace.shape, dev, 0)
    return workspace


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, scaling: str | None = None,
               factor: float = 1.0, original_positions: int = 4096, beta_fast: float = 32.0,
               beta_slow: float = 1.0, device="cuda") -> torch.Tensor:
    """The fp32 [max_positions, rot_dim] table of ``rope_append``: cosines, then sines, of
    p * base^(-2j / rot_dim), computed in 64 bits.

    ``scaling`` stretches it by ``factor`` for contexts longer than ``original_positions``:
    "linear" divides every frequency; "base" raises the base to base * factor^(r / (r - 2)),
    which leaves the highest frequency and divides the lowest by the factor; "ramp" leaves the
    frequencies that turn beta_fast times or more within the original context, divides those
    that turn beta_slow times or less, blends linearly between (in the pair's index) and
    multiplies the table by 0.1 ln(factor) + 1.
    """
    if rot_dim <= 0 or rot_dim % 16 or rot_dim > HEAD_DIM:
        raise ValueError(f"rot_dim must be a multiple of 16 in [16, {HEAD_DIM}], got {rot_dim}")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    amp = 1.0
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    j = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    inv = base ** (-2.0 * j / rot_dim)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "ramp":
        # the pair that turns b times within the original context
        pair = lambda b: rot_dim * math.log(original_positions / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = math.ceil(pair(beta_slow))     # may lie past the last pair, which then keeps a part
        slow = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        inv = inv * (1.0 - slow) + inv / factor * slow
        amp = 0.1 * math.log(factor) + 1.0
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos() * amp, a.sin() * amp), 1).float()


def add_rms_norm(x, residual, weight, eps: float = 1e-6, want: str = "bf16", group: int = 128,
                 residual_out=None, y=None, y8=None, y_scale=None, stream=None):
    """Run ``kda_add_rms_norm``: s = x + residual, y = s * (mean(s^2) + eps)^(-1/2) * weight.

    x: bf16 [T, C] (rows may be strided); residual: bf16 or fp32 [T, C], or None (s = x);
    weight: bf16 or fp32 [C].  want: "bf16" (y), "fp8" (y8 and y_scale) or "both"; y8 is
    float8_e4m3fn [T, C] with y_scale fp32 [T, ceil(C / 128)] (group 128) or [T, 1] (group 0).
    residual_out may be residual (the update is then in place).  Returns
    (residual_out, y, y8, y_scale) with None for what was not asked for.
    """
    if residual_out is None and y is None and y8 is None and y_scale is None and stream is None:
        done = (_native or _load_native()).add_rms_norm(x, residual, weight, eps, want, group)
        if done.__class__ is tuple:
            return done
        if done is not None:
            raise KDAError(done, "kda_add_rms_norm")
    dev = _need_cuda(x, "x")
    place = _elsewhere(stream, x)
    if place is not None:
        return _within(place, add_rms_norm, (residual_out, y, y8, y_scale), x, residual, weight, eps,
                          want, group, residual_out, y, y8, y_scale)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be 2-D")
    T, C = shape
    ldx = _check(x, "x", _HALF, shape, dev)
    _check(weight, "weight", _EITHER, (C,), dev, 0)
    ldr = lds = ldy = ldy8 = C
    r_ptr = s_ptr = y_ptr = y8_ptr = sc_ptr = None
    r_kind = STATE_BF16
    if residual is not None:
        ldr = _check(residual, "residual", _EITHER, shape, dev)
        r_ptr = residual.data_ptr()
        if residual.dtype is _F32:
            r_kind = STATE_F32
        if residual_out is None:
            residual_out = torch.empty_like(residual, memory_format=_DENSE)
        else:
            lds = _check(residual_out, "residual_out", (residual.dtype,), shape, dev)
        s_ptr = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    if want == "fp8":
        if y is not None:
            raise ValueError("y is not written with want='fp8'")
    else:
        if y is None:
            y = torch.empty_like(x, memory_format=_DENSE)
        else:
            ldy = _check(y, "y", _HALF, shape, dev)
        y_ptr = y.data_ptr()
    if want != "bf16":
        if want not in ("fp8", "both"):
            raise ValueError(f"want must be 'bf16', 'fp8' or 'both', got {want!r}")
        groups = -(-C // 128) if group == 128 else 1
        if y8 is None:
            y8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        else:
            ldy8 = _check(y8, "y8", _BYTES, shape, dev)
        if y_scale is None:
            y_scale = torch.empty((T, groups), dtype=_F32, device=dev)
        else:
            _check(y_scale, "y_scale", _FLOAT, (T, groups), dev, 0)
        y8_ptr, sc_ptr = y8.data_ptr(), y_scale.data_ptr()
    elif y8 is not None or y_scale is not None:
        raise ValueError("y8 and y_scale are not written with want='bf16'")
    group = _i32(group, "group")
    rc = lib().kda_add_rms_norm(
        x.data_ptr(), ldx, r_ptr, ldr, r_kind, weight.data_ptr(),
        STATE_F32 if weight.dtype is _F32 else STATE_BF16, eps, s_ptr, lds, y_ptr, ldy, y8_ptr, ldy8,
        sc_ptr, group, T, C, _stream(stream, dev))
    if rc != OK:
        raise KDAError(rc, "kda_add_rms_norm")
    return residual_out, y, y8, y_scale


def rope_append(q, k, v, rope, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens,
                cu_seqlens, interleaved: bool = False, positions=None, q_out=None, workspace=None,
                stream=None):
    """Run ``kda_rope_append``: rotate the new queries and keys, append the new keys and values.

    q: bf16 [T, heads, 128] or None; k, v: bf16 [T, kv_heads, 128] (tokens may be strided, e.g.
    column ranges of one fused projection); rope: fp32 [rows, rot_dim] (``rope_table``) or None
    for no rotation; cu_seqlens: int32 [num_seqs + 1]; positions: int32 [T] table rows, or None
    for the cache positions.  The cache tensors are updated in place.  Returns q_out (None
    without q).  workspace: uint8, at least 256 bytes, zero-filled once (device status).
    """
    if q_out is None and stream is None:
        done = (_native or _load_native()).rope_append(
            q, k, v, rope, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
            interleaved, positions, workspace)
        if done.__class__ is int:
            raise KDAError(done, "kda_rope_append")
        if done is not None:
            return done
    dev = _need_cuda(k, "k")
    place = _elsewhere(stream, k)
    if place is not None:
        return _within(place, rope_append, (q_out,), q, k, v, rope, k_cache, v_cache, k_scale, v_scale,
                          block_table, kv_lens, cu_seqlens, interleaved, positions, q_out, workspace)
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k must be [T, kv_heads, 128]")
    T, heads, d = shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    N = cu_seqlens.numel() - 1
    k_row = _check(k, "k", _HALF, shape, dev)
    v_row = _check(v, "v", _HALF, shape, dev)
    q_ptr = qo_ptr = rope_ptr = pos_ptr = None
    q_row = qo_row = rows = rot = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, heads, 128]")
        heads = q.shape[1]
        q_shape = (T, heads, HEAD_DIM)
        q_row = _check(q, "q", _HALF, q_shape, dev)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=_DENSE)
            qo_row = heads * HEAD_DIM
        else:
            qo_row = _check(q_out, "q_out", _HALF, q_shape, dev)
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(cu_seqlens, "cu_seqlens", _INT, (N + 1,), dev, 0)
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [rows, rot_dim]")
        rows, rot = rope.shape
        _check(rope, "rope", _FLOAT, rope.shape, dev, 0)
        rope_ptr = rope.data_ptr()
    if positions is not None:
        _check(positions, "positions", _INT, (T,), dev, 0)
        pos_ptr = positions.data_ptr()
    c, hk = _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, N, dev)
    if hk != shape[1]:
        raise ValueError(f"k has {shape[1]} heads, the cache {hk}")
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_rope_append(
        q_ptr, q_row, k.data_ptr(), k_row, v.data_ptr(), v_row, rope_ptr, rows, rot,
        1 if interleaved else 0, pos_ptr, qo_ptr, qo_row, c, cu_seqlens.data_ptr(),
        workspace.data_ptr(), _stream(stream, dev), T, N, heads, workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_rope_append")
    return q_out


def attention_workspace_size(num_seqs: int, heads: int, kv_heads: int, max_q_len: int) -> int:
    return int(lib().kda_attention_workspace_size(
        _i32(int(num_seqs), "num_seqs"), _i32(int(heads), "heads"), _i32(int(kv_heads), "kv_heads"),
        _i32(int(max_q_len), "max_q_len")))


def alloc_attention_workspace(num_seqs: int, heads: int, kv_heads: int, max_q_len: int,
                              device=None) -> torch.Tensor:
    """A zero-filled uint8 workspace for ``cached_attention``."""
    n = attention_workspace_size(num_seqs, heads, kv_heads, max_q_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def cached_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                     scale: float, max_q_len: int, softcap: float = 0.0, window: int = 0,
                     out=None, lse=False, workspace=None, stream=None):
    """Run ``kda_cached_attention``: causal attention of the new queries over the cache.

    q: bf16 [T, heads, 128]; cu_seqlens: int32 [num_seqs + 1]; max_q_len: an upper bound of one
    sequence's new tokens.  softcap > 0 caps the scores by softcap * tanh(s / softcap); window >
    0 limits each query to the last ``window`` positions, its own included.  lse: False, True
    (allocate fp32 [T, heads]) or a tensor.  workspace: ``alloc_attention_workspace`` of the same
    sizes or larger ones.  Returns (out, lse or None).
    """
    if out is None and stream is None:
        done = (_native or _load_native()).cached_attention(
            q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, scale, max_q_len,
            softcap, window, lse, workspace)
        if done.__class__ is tuple:
            return done
        if done is not None:
            raise KDAError(done, "kda_cached_attention")
    dev = _need_cuda(q, "q")
    place = _elsewhere(stream, q)
    if place is not None:
        return _within(place, cached_attention, (out, lse if isinstance(lse, torch.Tensor) else None), q,
                          k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, scale,
                          max_q_len, softcap, window, out, lse, workspace)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T, heads, 128]")
    T, heads, d = shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    N = cu_seqlens.numel() - 1
    window, max_q_len = _i32(window, "window"), _i32(max_q_len, "max_q_len")
    q_row = _check(q, "q", _HALF, shape, dev)
    _check(cu_seqlens, "cu_seqlens", _INT, (N + 1,), dev, 0)
    c, hk = _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, N, dev)
    out_row = heads * HEAD_DIM
    if out is None:
        out = torch.empty_like(q, memory_format=_DENSE)
    else:
        out_row = _check(out, "out", _HALF, shape, dev)
    lse_ptr = None
    if lse is False:
        lse = None
    else:
        if lse is True:
            lse = torch.empty((T, heads), dtype=_F32, device=dev)
        else:
            _check(lse, "lse", _FLOAT, (T, heads), dev, 0)
        lse_ptr = lse.data_ptr()
    if workspace is None:
        # (this call's alone: its status words are zeroed, the rest is written before it is read)
        workspace = torch.empty(max(attention_workspace_size(N, heads, hk, max_q_len), 256),
                                dtype=torch.uint8, device=dev)
        workspace[:256].zero_()
    else:
        _check(workspace, "workspace", _UINT8, workspace.shape, dev, 0)
    rc = lib().kda_cached_attention(
        q.data_ptr(), q_row, c, cu_seqlens.data_ptr(), scale, softcap, window, out.data_ptr(), out_row,
        lse_ptr, workspace.data_ptr(), _stream(stream, dev), T, N, heads, max_q_len, workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_cached_attention")
    return out, lse
