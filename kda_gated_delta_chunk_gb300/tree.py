"""Trees of drafted tokens: what a step needs of them, the KDA recurrence along their branches, and
what acceptance does to state and cache.

The calls of ``include/kda.h``'s section on trees, on torch tensors; marshalling only.  A batch's new
tokens are packed by cu_seqlens, at most 64 a sequence, and

    parents    int32 [T]: the index, among its sequence's new tokens, of the one that token t follows,
               -1 for one that follows the cached text; parents come before their children

A step appends its nodes to the cache in their order (``rope_append`` with ``positions``), attends
with ``tree_attention``, and keeps the branch that was accepted.
"""
from __future__ import annotations

import torch

from . import ERR_INVALID_ARG, HEAD_DIM, KDAError, OK, STATE_BF16, STATE_F32, _elsewhere, _within, lib
from .layer import _EITHER, _F32, _FLOAT, _HALF, _I32, _INT, _MASK, _cache, _check, _i32, _need_cuda, _status_workspace, _stream, native


def _batch(parents, cu_seqlens, dev):
    """Total tokens and number of sequences of a batch of trees."""
    if parents.dim() != 1:
        raise ValueError("parents must be [T]")
    _check(parents, "parents", _INT, parents.shape, dev, 0)
    n = cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", _INT, (n + 1,), dev, 0)
    return parents.shape[0], n


def tree_plan(parents, cu_seqlens, kv_lens, max_q_len: int, mask=None, positions=None, workspace=None,
              stream=None):
    """Run ``kda_tree_plan``: the nodes' masks and positions, once for all layers of a step.

    parents: int32 [T]; cu_seqlens: int32 [num_seqs + 1]; kv_lens: int32 [num_seqs], the nodes
    included; max_q_len: an upper bound of one sequence's nodes, at most 64.  Returns (mask, positions):
    int64 [T] for ``tree_attention`` and int32 [T] for ``rope_append``.
    """
    if mask is None and positions is None and stream is None:
        done = native().tree_plan(parents, cu_seqlens, kv_lens, max_q_len, workspace)
        if done.__class__ is tuple:
            return done
        if done is not None:
            raise KDAError(done, "kda_tree_plan")
    dev = _need_cuda(parents, "parents")
    place = _elsewhere(stream, parents)
    if place is not None:
        return _within(place, tree_plan, (mask, positions), parents, cu_seqlens, kv_lens, max_q_len, mask,
                       positions, workspace)
    T, N = _batch(parents, cu_seqlens, dev)
    _check(kv_lens, "kv_lens", _INT, (N,), dev, 0)
    if mask is None:
        mask = torch.empty(T, dtype=torch.int64, device=parents.device)
    else:
        _check(mask, "mask", _MASK, (T,), dev, 0)
    if positions is None:
        positions = torch.empty(T, dtype=_I32, device=parents.device)
    else:
        _check(positions, "positions", _INT, (T,), dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_tree_plan(parents.data_ptr(), cu_seqlens.data_ptr(), kv_lens.data_ptr(), mask.data_ptr(),
                             positions.data_ptr(), workspace.data_ptr(), _stream(stream, dev), T, N,
                             _i32(max_q_len, "max_q_len"), workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_tree_plan")
    return mask, positions


def _rows(t, name, shape, dev):
    """Token stride of a bf16 [T, heads, 128] (or [T, heads]) tensor, tokens strided, the rest dense."""
    return _check(t, name, _HALF, shape, dev)


def _state(initial_state, state_dtype, n, heads, dev):
    """Pointer, kind and dtype of the state before the tree."""
    if initial_state is None:
        dtype = _F32 if state_dtype is None else state_dtype
    else:
        dtype = initial_state.dtype if state_dtype is None else state_dtype
        _check(initial_state, "initial_state", (dtype,), (n, heads, HEAD_DIM, HEAD_DIM), dev, 0)
    if dtype not in _EITHER:
        raise TypeError("state dtype must be float32 or bfloat16")
    return (None if initial_state is None else initial_state.data_ptr(),
            STATE_F32 if dtype is _F32 else STATE_BF16, dtype)


def _heads(k, dev):
    if k.dim() != 3:
        raise ValueError("k must be [T, heads, 128]")
    T, H, d = k.shape
    if d != HEAD_DIM:
        raise KDAError(ERR_INVALID_ARG, f"head_dim {d} (only {HEAD_DIM} is supported)")
    return T, H


def tree_recurrent_fwd(q, k, v, g, beta, A_log, dt_bias, lower_bound: float, scale: float, initial_state,
                       cu_seqlens, parents, max_q_len: int, out=None, u=None, state_dtype=None, workspace=None,
                       stream=None):
    """Run ``kda_tree_recurrent_fwd``: the KDA recurrence along the branches of drafted trees.

    q, k, v, g: bf16 [T, heads, 128] and beta: bf16 [T, heads] (tokens may be strided, e.g. column ranges of
    one fused projection); A_log, dt_bias, initial_state and cu_seqlens as in ``recurrent_fwd``; parents:
    int32 [T]; max_q_len: an upper bound of one sequence's nodes, at most 64.  The state is read
    only.  Returns (out, u): bf16 [T, heads, 128], and fp32 [T, heads, 128] for ``tree_commit``.
    """
    if out is None and u is None and state_dtype is None and stream is None:
        done = native().tree_recurrent_fwd(q, k, v, g, beta, A_log, dt_bias, lower_bound, scale, initial_state,
                                           cu_seqlens, parents, max_q_len, workspace)
        if done.__class__ is tuple:
            return done
        if done is not None:
            raise KDAError(done, "kda_tree_recurrent_fwd")
    dev = _need_cuda(k, "k")
    place = _elsewhere(stream, k)
    if place is not None:
        return _within(place, tree_recurrent_fwd, (out, u), q, k, v, g, beta, A_log, dt_bias, lower_bound, scale,
                       initial_state, cu_seqlens, parents, max_q_len, out, u, state_dtype, workspace)
    T, H = _heads(k, dev)
    shape = k.shape
    nodes, N = _batch(parents, cu_seqlens, dev)
    if nodes != T:
        raise ValueError(f"parents has {nodes} entries, k {T} tokens")
    strides = [_rows(t, name, shape, dev) for t, name in ((q, "q"), (k, "k"), (v, "v"), (g, "g"))]
    beta_row = _rows(beta, "beta", (T, H), dev)
    _check(A_log, "A_log", _FLOAT, (H,), dev, 0)
    _check(dt_bias, "dt_bias", _FLOAT, (H, HEAD_DIM), dev, 0)
    state, kind, _ = _state(initial_state, state_dtype, N, H, dev)
    if out is None:
        out = torch.empty(shape, dtype=k.dtype, device=k.device)
    else:
        _check(out, "out", _HALF, shape, dev, 0)
    if u is None:
        u = torch.empty(shape, dtype=_F32, device=k.device)
    else:
        _check(u, "u", _FLOAT, shape, dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_tree_recurrent_fwd(
        q.data_ptr(), strides[0], k.data_ptr(), strides[1], v.data_ptr(), strides[2], g.data_ptr(), strides[3],
        beta.data_ptr(), beta_row, A_log.data_ptr(), dt_bias.data_ptr(), lower_bound, scale, state, kind,
        cu_seqlens.data_ptr(), parents.data_ptr(), out.data_ptr(), u.data_ptr(), workspace.data_ptr(),
        _stream(stream, dev), T, N, H, _i32(max_q_len, "max_q_len"), workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_tree_recurrent_fwd")
    return out, u


def tree_commit(k, g, A_log, dt_bias, lower_bound: float, initial_state, cu_seqlens, parents, u, accepted,
                max_q_len: int, final_state=None, state_dtype=None, workspace=None, stream=None):
    """Run ``kda_tree_commit``: the state after each tree's accepted branch.

    k, g, A_log, dt_bias, lower_bound, initial_state, cu_seqlens, parents and max_q_len as given to
    ``tree_recurrent_fwd``, u as it returned it; accepted: int32 [num_seqs], the last accepted node of
    each sequence (-1: none, its state stays).  final_state may be initial_state (the update is then
    in place).  Returns final_state.
    """
    if state_dtype is None and stream is None:
        done = native().tree_commit(k, g, A_log, dt_bias, lower_bound, initial_state, cu_seqlens, parents, u,
                                    accepted, max_q_len, final_state, workspace)
        if done.__class__ is int:
            raise KDAError(done, "kda_tree_commit")
        if done is not None:
            return done
    dev = _need_cuda(k, "k")
    place = _elsewhere(stream, k)
    if place is not None:
        return _within(place, tree_commit, (final_state,), k, g, A_log, dt_bias, lower_bound, initial_state,
                       cu_seqlens, parents, u, accepted, max_q_len, final_state, state_dtype, workspace)
    T, H = _heads(k, dev)
    nodes, N = _batch(parents, cu_seqlens, dev)
    if nodes != T:
        raise ValueError(f"parents has {nodes} entries, k {T} tokens")
    k_row, g_row = _rows(k, "k", k.shape, dev), _rows(g, "g", k.shape, dev)
    _check(A_log, "A_log", _FLOAT, (H,), dev, 0)
    _check(dt_bias, "dt_bias", _FLOAT, (H, HEAD_DIM), dev, 0)
    _check(u, "u", _FLOAT, k.shape, dev, 0)
    _check(accepted, "accepted", _INT, (N,), dev, 0)
    if initial_state is None and state_dtype is None and final_state is not None:
        state_dtype = final_state.dtype
    state, kind, dtype = _state(initial_state, state_dtype, N, H, dev)
    if final_state is None:
        final_state = torch.empty((N, H, HEAD_DIM, HEAD_DIM), dtype=dtype, device=k.device)
    else:
        _check(final_state, "final_state", (dtype,), (N, H, HEAD_DIM, HEAD_DIM), dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_tree_commit(
        k.data_ptr(), k_row, g.data_ptr(), g_row, A_log.data_ptr(), dt_bias.data_ptr(), lower_bound, state,
        final_state.data_ptr(), kind, cu_seqlens.data_ptr(), parents.data_ptr(), u.data_ptr(),
        accepted.data_ptr(), workspace.data_ptr(), _stream(stream, dev), T, N, H, _i32(max_q_len, "max_q_len"),
        workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_tree_commit")
    return final_state


def cache_accept(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, parents, accepted,
                 max_q_len: int, lens_out=None, workspace=None, stream=None):
    """Run ``kda_cache_accept``: move each tree's accepted branch together in one layer's cache.

    The cache and its indexes as for ``tree_attention``; accepted: int32 [num_seqs], the last accepted
    node of each sequence (-1: none).  The cache is updated in place.  Returns lens_out, int32
    [num_seqs]: the cached tokens from there on (a tensor of its own: every layer's call reads kv_lens).
    """
    if lens_out is None and stream is None:
        done = native().cache_accept(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                     parents, accepted, max_q_len, workspace)
        if done.__class__ is int:
            raise KDAError(done, "kda_cache_accept")
        if done is not None:
            return done
    dev = _need_cuda(k_cache, "k_cache")
    place = _elsewhere(stream, k_cache)
    if place is not None:
        return _within(place, cache_accept, (lens_out,), k_cache, v_cache, k_scale, v_scale, block_table, kv_lens,
                       cu_seqlens, parents, accepted, max_q_len, lens_out, workspace)
    T, N = _batch(parents, cu_seqlens, dev)
    c, _ = _cache(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, N, dev)
    _check(accepted, "accepted", _INT, (N,), dev, 0)
    if lens_out is None:
        lens_out = torch.empty(N, dtype=_I32, device=k_cache.device)
    else:
        _check(lens_out, "lens_out", _INT, (N,), dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_cache_accept(c, cu_seqlens.data_ptr(), parents.data_ptr(), accepted.data_ptr(),
                                lens_out.data_ptr(), workspace.data_ptr(), _stream(stream, dev), T, N,
                                _i32(max_q_len, "max_q_len"), workspace.numel())
    if rc != OK:
        raise KDAError(rc, "kda_cache_accept")
    return lens_out
