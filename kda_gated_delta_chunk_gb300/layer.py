"""The full-attention layer's operators: residual norm, rotary append to a paged 8-bit cache,
attention over that cache.

The calls of ``include/kda.h``'s section on the full-attention layer, on torch tensors; like
the rest of the binding, marshalling only.  A cache is four tensors and two indexes:

    k_cache, v_cache   float8_e4m3fn (or uint8) [pages, kv_heads, page_size, 128], any strides
                       that are multiples of 16 with the channels dense
    k_scale, v_scale   fp32 [pages, kv_heads]
    block_table        int32 [num_seqs, max_blocks]: the pages of each sequence, in order
    kv_lens            int32 [num_seqs]: cached tokens, the step's new ones included
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (ERR_INVALID_ARG, HEAD_DIM, KDAError, OK, STATE_BF16, STATE_F32, lib)

_BF16, _F32 = torch.bfloat16, torch.float32
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_HALF, _EITHER = (_BF16,), (_BF16, _F32)
_FLOAT = (_F32,)
_INT = (torch.int32,)
# the current stream's handle without a Stream object around it (a call's host time counts in decode)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("kv_lens", ctypes.c_void_p)]


def _check(t, name, dtypes, shape, dev, dense_from=1):
    """Type, device and shape; dimensions from ``dense_from`` on are dense."""
    if (isinstance(t, torch.Tensor) and t.device == dev and t.dtype in dtypes and t.shape == shape
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
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


def _row_stride(t, dense):
    return t.stride(0) if t.shape[0] > 1 else dense


def _stream(stream, dev):
    return stream.cuda_stream if stream is not None else _raw_stream(dev.index)


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, num_seqs, dev):
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, 128]")
    pages, hk, page, d = shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    _check(k_cache, "k_cache", _BYTES, shape, dev, 3)
    _check(v_cache, "v_cache", _BYTES, shape, dev, 3)
    st, sc = k_cache.stride(), k_scale.stride()
    if v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same strides")
    _check(k_scale, "k_scale", _FLOAT, (pages, hk), dev)
    _check(v_scale, "v_scale", _FLOAT, (pages, hk), dev)
    if v_scale.stride() != sc:
        raise ValueError("k_scale and v_scale must have the same strides")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [num_seqs, max_blocks]")
    blocks = block_table.shape[1]
    _check(block_table, "block_table", _INT, (num_seqs, blocks), dev)
    _check(kv_lens, "kv_lens", _INT, (num_seqs,), dev, 0)
    # dimensions of one element take the dense stride: torch leaves theirs arbitrary
    tok = st[2] if page > 1 else HEAD_DIM
    head = st[1] if hk > 1 else page * tok
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                  st[0] if pages > 1 else hk * head, head, tok, sc[0] if pages > 1 else hk, pages,
                  page, hk, blocks, block_table.data_ptr(), _row_stride(block_table, blocks),
                  kv_lens.data_ptr())


def _status_workspace(workspace, dev):
    if workspace is None:
        return torch.zeros(256, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", (torch.uint8,), workspace.shape, dev, 0)
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
        hi = min(math.ceil(pair(beta_slow)), rot_dim // 2 - 1)
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
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if want not in ("bf16", "fp8", "both"):
        raise ValueError(f"want must be 'bf16', 'fp8' or 'both', got {want!r}")
    dev = x.device
    T, C = x.shape
    _check(x, "x", _HALF, x.shape, None)
    _check(weight, "weight", _EITHER, (C,), dev, 0)
    if residual is not None:
        _check(residual, "residual", _EITHER, x.shape, dev)
        if residual_out is None:
            residual_out = torch.empty((T, C), dtype=residual.dtype, device=dev)
        else:
            _check(residual_out, "residual_out", (residual.dtype,), x.shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    if want == "fp8":
        if y is not None:
            raise ValueError("y is not written with want='fp8'")
    elif y is None:
        y = torch.empty((T, C), dtype=_BF16, device=dev)
    else:
        _check(y, "y", _HALF, x.shape, dev)
    if want == "bf16":
        if y8 is not None or y_scale is not None:
            raise ValueError("y8 and y_scale are not written with want='bf16'")
    else:
        groups = -(-C // 128) if group == 128 else 1
        if y8 is None:
            y8 = torch.empty((T, C), dtype=torch.float8_e4m3fn, device=dev)
        else:
            _check(y8, "y8", _BYTES, x.shape, dev)
        if y_scale is None:
            y_scale = torch.empty((T, groups), dtype=_F32, device=dev)
        else:
            _check(y_scale, "y_scale", _FLOAT, (T, groups), dev, 0)
    has_r, has_y, has_8 = residual is not None, y is not None, y8 is not None
    rc = lib().kda_add_rms_norm(
        x.data_ptr(), _row_stride(x, C), residual.data_ptr() if has_r else None,
        _row_stride(residual, C) if has_r else C,
        STATE_F32 if has_r and residual.dtype == _F32 else STATE_BF16, weight.data_ptr(),
        STATE_F32 if weight.dtype == _F32 else STATE_BF16, eps,
        residual_out.data_ptr() if has_r else None, _row_stride(residual_out, C) if has_r else C,
        y.data_ptr() if has_y else None, _row_stride(y, C) if has_y else C,
        y8.data_ptr() if has_8 else None, _row_stride(y8, C) if has_8 else C,
        y_scale.data_ptr() if has_8 else None, group, T, C, _stream(stream, dev))
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
    if k.dim() != 3:
        raise ValueError("k must be [T, kv_heads, 128]")
    dev = k.device
    T, hk, d = k.shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    N = cu_seqlens.numel() - 1
    _check(k, "k", _HALF, k.shape, None)
    _check(v, "v", _HALF, k.shape, dev)
    heads = hk
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, heads, 128]")
        heads = q.shape[1]
        _check(q, "q", _HALF, (T, heads, d), dev)
        if q_out is None:
            q_out = torch.empty((T, heads, d), dtype=_BF16, device=dev)
        else:
            _check(q_out, "q_out", _HALF, (T, heads, d), dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(cu_seqlens, "cu_seqlens", _INT, (N + 1,), dev, 0)
    rows = rot = 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [rows, rot_dim]")
        rows, rot = rope.shape
        _check(rope, "rope", _FLOAT, rope.shape, dev, 0)
    if positions is not None:
        _check(positions, "positions", _INT, (T,), dev, 0)
    c = _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, N, dev)
    if c.kv_heads != hk:
        raise ValueError(f"k has {hk} heads, the cache {c.kv_heads}")
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_rope_append(
        None if q is None else q.data_ptr(), heads * d if q is None else _row_stride(q, heads * d),
        k.data_ptr(), _row_stride(k, hk * d), v.data_ptr(), _row_stride(v, hk * d),
        None if rope is None else rope.data_ptr(), rows, rot, int(bool(interleaved)),
        None if positions is None else positions.data_ptr(),
        None if q is None else q_out.data_ptr(), heads * d if q is None else _row_stride(q_out, heads * d),
        ctypes.byref(c), cu_seqlens.data_ptr(), workspace.data_ptr(), _stream(stream, dev), T, N,
        heads, workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_rope_append")
    return q_out


def attention_workspace_size(num_seqs: int, heads: int, kv_heads: int, max_q_len: int) -> int:
    return int(lib().kda_attention_workspace_size(int(num_seqs), int(heads), int(kv_heads),
                                                  int(max_q_len)))


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
    if q.dim() != 3:
        raise ValueError("q must be [T, heads, 128]")
    dev = q.device
    T, heads, d = q.shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    N = cu_seqlens.numel() - 1
    _check(q, "q", _HALF, q.shape, None)
    _check(cu_seqlens, "cu_seqlens", _INT, (N + 1,), dev, 0)
    c = _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, N, dev)
    if out is None:
        out = torch.empty((T, heads, d), dtype=_BF16, device=dev)
    else:
        _check(out, "out", _HALF, q.shape, dev)
    if lse is True:
        lse = torch.empty((T, heads), dtype=_F32, device=dev)
    elif lse is False:
        lse = None
    else:
        _check(lse, "lse", _FLOAT, (T, heads), dev, 0)
    if workspace is None:
        workspace = alloc_attention_workspace(N, heads, c.kv_heads, max_q_len, dev)
    else:
        _check(workspace, "workspace", (torch.uint8,), workspace.shape, dev, 0)
    rc = lib().kda_cached_attention(
        q.data_ptr(), _row_stride(q, heads * d), ctypes.byref(c), cu_seqlens.data_ptr(), scale,
        softcap, window, out.data_ptr(), _row_stride(out, heads * d),
        None if lse is None else lse.data_ptr(), workspace.data_ptr(), _stream(stream, dev), T, N,
        heads, max_q_len, workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_cached_attention")
    return out, lse
