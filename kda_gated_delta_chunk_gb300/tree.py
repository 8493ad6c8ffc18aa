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

from . import KDAError, OK, _elsewhere, _within, lib
from .layer import _I32, _INT, _MASK, _cache, _check, _i32, _need_cuda, _status_workspace, _stream


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


def cache_accept(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, parents, accepted,
                 max_q_len: int, lens_out=None, workspace=None, stream=None):
    """Run ``kda_cache_accept``: move each tree's accepted branch together in one layer's cache.

    The cache and its indexes as for ``tree_attention``; accepted: int32 [num_seqs], the last accepted
    node of each sequence (-1: none).  The cache is updated in place.  Returns lens_out, int32
    [num_seqs]: the cached tokens from there on (a tensor of its own: every layer's call reads kv_lens).
    """
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
