"""The pages of a paged cache on the device: given back, reserved, shared by forked sequences, copied.

The calls of ``include/kda.h``'s section on pages, on torch tensors; marshalling only.  A pool is

    refs          int32 [pages]: the rows that hold each page; 0: free
    block_table   int32 [rows, max_blocks]: the pages of each sequence, in order, -1 behind them
    kv_lens       int32 [rows]

updated in place; who needs pages gets the lowest free ones, in the order of rows and blocks.
block_table and kv_lens are those of ``rope_append`` and the attention calls.  A page that more than one row holds
is for reading: ``reserve_pages`` looks at the counts before ``rope_append`` and ``cache_accept`` write.
"""
from __future__ import annotations

import torch

from . import KDAError, OK, _elsewhere, _within, lib
from .layer import _I32, _INT, _cache, _check, _i32, _need_cuda, _status_workspace, _stream, native


def _pool(refs, block_table, kv_lens, page_size, dev):
    """The arguments of a pool."""
    if refs.dim() != 1:
        raise ValueError("refs must be [pages]")
    _check(refs, "refs", _INT, refs.shape, dev, 0)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_blocks]")
    rows, blocks = block_table.shape
    stride = _check(block_table, "block_table", _INT, block_table.shape, dev)
    _check(kv_lens, "kv_lens", _INT, (rows,), dev, 0)
    return (refs.data_ptr(), refs.shape[0], block_table.data_ptr(), stride if rows > 1 else blocks, rows, blocks,
            kv_lens.data_ptr(), _i32(page_size, "page_size"))


def _list(t, name, dev):
    if t.dim() != 1:
        raise ValueError(f"{name} must be one-dimensional")
    _check(t, name, _INT, t.shape, dev, 0)
    return t.shape[0]


def free_pages(refs, block_table, kv_lens, page_size: int, rows=None, workspace=None, stream=None):
    """Run ``kda_pages_free``: give pages back to the pool.

    rows: None (every row gives back the pages beyond its kv_lens) or int32 [m] (those rows end: all
    their pages go back, their kv_lens become 0).
    """
    if stream is None:
        done = native().free_pages(refs, block_table, kv_lens, page_size, rows, workspace)
        if done is True:
            return
        if done is not None:
            raise KDAError(done, "kda_pages_free")
    dev = _need_cuda(refs, "refs")
    place = _elsewhere(stream, refs)
    if place is not None:
        return _within(place, free_pages, (), refs, block_table, kv_lens, page_size, rows, workspace)
    pool = _pool(refs, block_table, kv_lens, page_size, dev)
    num = 0 if rows is None else _list(rows, "rows", dev)
    if rows is not None and num == 0:
        return
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_pages_free(*pool, None if rows is None else rows.data_ptr(), num, workspace.data_ptr(),
                              workspace.numel(), _stream(stream, dev))
    if rc != OK:
        raise KDAError(rc, "kda_pages_free")


def reserve_pages(refs, block_table, kv_lens, new_tokens, page_size: int, workspace=None, stream=None):
    """Run ``kda_pages_reserve``: pages for new_tokens (int32 [rows]) more tokens of each row.

    A row whose new tokens would go into a page that other rows hold as well (its kv_lens was set back into a
    shared one) is reported and gets none; a fork of it has a page of its own there.
    """
    if stream is None:
        done = native().reserve_pages(refs, block_table, kv_lens, new_tokens, page_size, workspace)
        if done is True:
            return
        if done is not None:
            raise KDAError(done, "kda_pages_reserve")
    dev = _need_cuda(refs, "refs")
    place = _elsewhere(stream, refs)
    if place is not None:
        return _within(place, reserve_pages, (), refs, block_table, kv_lens, new_tokens, page_size, workspace)
    pool = _pool(refs, block_table, kv_lens, page_size, dev)
    _check(new_tokens, "new_tokens", _INT, kv_lens.shape, dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_pages_reserve(*pool, new_tokens.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                 _stream(stream, dev))
    if rc != OK:
        raise KDAError(rc, "kda_pages_reserve")


def fork_pages(refs, block_table, kv_lens, src, dst, page_size: int, from_pages=None, to_pages=None,
               workspace=None, stream=None):
    """Run ``kda_pages_fork``: rows dst (int32 [m]) become copies of rows src (int32 [m]).

    Whole pages are shared.  Returns (from_pages, to_pages), int32 [m] for ``copy_pages`` on every layer's
    cache: a partly filled last page and the one to copy it to, -1 where there is none.  The rows of dst
    hold no pages before (``free_pages``), and none is a source.  Where the pool has too few pages
    (ERR_OUT_OF_PAGES), a row without its last page is to be ended, or its kv_lens set down to its whole pages.
    """
    if from_pages is None and to_pages is None and stream is None:
        done = native().fork_pages(refs, block_table, kv_lens, src, dst, page_size, workspace)
        if done.__class__ is tuple:
            return done
        if done is not None:
            raise KDAError(done, "kda_pages_fork")
    dev = _need_cuda(refs, "refs")
    place = _elsewhere(stream, refs)
    if place is not None:
        return _within(place, fork_pages, (from_pages, to_pages), refs, block_table, kv_lens, src, dst, page_size,
                       from_pages, to_pages, workspace)
    pool = _pool(refs, block_table, kv_lens, page_size, dev)
    num = _list(src, "src", dev)
    _check(dst, "dst", _INT, (num,), dev, 0)
    if from_pages is None:
        from_pages = torch.empty(num, dtype=_I32, device=refs.device)
    else:
        _check(from_pages, "from_pages", _INT, (num,), dev, 0)
    if to_pages is None:
        to_pages = torch.empty(num, dtype=_I32, device=refs.device)
    else:
        _check(to_pages, "to_pages", _INT, (num,), dev, 0)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_pages_fork(*pool, src.data_ptr(), dst.data_ptr(), num, from_pages.data_ptr(),
                              to_pages.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _stream(stream, dev))
    if rc != OK:
        raise KDAError(rc, "kda_pages_fork")
    return from_pages, to_pages


def copy_pages(k_cache, v_cache, k_scale, v_scale, from_pages, to_pages, workspace=None, stream=None):
    """Run ``kda_pages_copy``: pages from_pages to pages to_pages (int32 [m]) of one layer's cache, with
    their scales; pairs with a negative page are left out."""
    if stream is None:
        done = native().copy_pages(k_cache, v_cache, k_scale, v_scale, from_pages, to_pages, workspace)
        if done is True:
            return
        if done is not None:
            raise KDAError(done, "kda_pages_copy")
    dev = _need_cuda(k_cache, "k_cache")
    place = _elsewhere(stream, k_cache)
    if place is not None:
        return _within(place, copy_pages, (), k_cache, v_cache, k_scale, v_scale, from_pages, to_pages, workspace)
    num = _list(from_pages, "from_pages", dev)
    _check(to_pages, "to_pages", _INT, (num,), dev, 0)
    # (the cache's tensors alone: an empty table and no lengths)
    c, _ = _cache(k_cache, v_cache, k_scale, v_scale, from_pages[:0].view(0, 1), from_pages[:0], 0, dev)
    workspace = _status_workspace(workspace, dev)
    rc = lib().kda_pages_copy(c, from_pages.data_ptr(), to_pages.data_ptr(), num, workspace.data_ptr(),
                              workspace.numel(), _stream(stream, dev))
    if rc != OK:
        raise KDAError(rc, "kda_pages_copy")
