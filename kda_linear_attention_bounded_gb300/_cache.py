"""torch binding of the calls around the paged cache (``include/kda.h``): rotary positions with the store into the
pages, forking and ending requests, compacting and copying pages, attention over prefixes that requests share.

Tensors are checked as in ``_hybrid``; a call runs with the tensors' device current, on the given stream or that device's
current one.
"""
from __future__ import annotations

import operator

from . import _binding as _b
from . import _hybrid as _h
from ._binding import KDA_OK, KdaError


def _raw(stream, x):
    return None if stream is None else _h._raw(stream, x)


def _workspace(workspace, x, name, stream, nbytes=None):
    return _h._new_workspace(_h._cuda(x, name), stream, nbytes) if workspace is None else workspace


def _done(rc, what):
    if rc != KDA_OK:
        raise KdaError(rc, what)


def rotary_to_pages(q, k, v, positions, slot_map, inv_freq, k_pages, v_pages, *, axes=None, interleaved=False, mscale=1.0,
                    out=None, workspace=None, stream=None):
    """``kda_rotary_to_pages``: the step's queries turned by their positions, its keys turned and stored into their
    pages with the values.

    q: bf16 ``[tokens, Hq, 128]``; k, v: bf16 ``[tokens, Hk, 128]`` (any token strides); positions: int32 ``[tokens]``, or
    ``[axes, tokens]`` with one row for each axis (time, height, width); slot_map: int64 ``[tokens]`` as
    :func:`step_tables` writes it (-1: a padding token, left out); inv_freq: fp32 ``[R / 2]`` frequencies, of which ``axes``
    (whole numbers, one a frequency; bytes save a conversion) says whose position each turns by.  ``interleaved``: the pairs are
    channels 2f, 2f + 1 instead of f, f + R / 2.  mscale: factor of the turned channels.  out: the turned queries, which
    may be q itself.  Returns ``out``."""
    if out is None:
        out = _h._rows_like(q, "q", stream)
    if axes is not None and axes.__class__ is not bytes:
        axes = bytes(map(operator.index, axes))
    workspace = _workspace(workspace, q, "q", stream)
    _done(_h._ext.rotary_to_pages(q, k, v, positions, slot_map, inv_freq, k_pages, v_pages, axes, bool(interleaved), mscale, out,
                                  workspace, _raw(stream, q)), "kda_rotary_to_pages")
    return out


def fork_requests(block_table, seq_lens, parents, children, free_pages, page_size, *, copy_src, copy_dst, pages_used,
                  workspace=None, stream=None):
    """``kda_fork_requests``: rows ``children`` of the table become copies of rows ``parents`` (int32 ``[forks]``; a
    negative one is padding).  Whole pages are shared, the rest of a page gets a page of its own from the front of
    free_pages (which ends at its first negative id, as :func:`release_requests` leaves it), with the copy to make in copy_src, copy_dst (int32 ``[forks]``, -1: none; :func:`copy_pages` takes them).
    seq_lens of the children and pages_used (int32 ``[1]``) are written.  :func:`copy_pages` also copies the recurrent states
    of a hybrid model's forked requests, with slots for pages."""
    workspace = _workspace(workspace, block_table, "block_table", stream)
    _done(_h._ext.fork_requests(block_table, seq_lens, parents, children, free_pages, page_size, copy_src, copy_dst, pages_used,
                                workspace, _raw(stream, block_table)), "kda_fork_requests")


def release_requests(block_table, seq_lens, rows, page_size, *, free_pages, num_free, workspace=None, stream=None):
    """``kda_release_requests``: the requests ``rows`` (int32; a negative one is padding) end, their seq_lens become 0, and
    free_pages (int32 ``[pages of the cache]``) is written anew: the pages that no row holds, ascending, then -1; num_free
    (int32 ``[1]``): how many."""
    workspace = _workspace(workspace, block_table, "block_table", stream)
    _done(_h._ext.release_requests(block_table, seq_lens, rows, page_size, free_pages, num_free, workspace,
                                   _raw(stream, block_table)), "kda_release_requests")


def compact_pages(block_table, seq_lens, page_size, *, new_table, copy_src, copy_dst, free_pages, num_free, workspace=None,
                  stream=None):
    """``kda_compact_pages``: the pages in use move to the first ids.  Written: new_table (``block_table`` itself or another
    of its shape), the copies that :func:`copy_pages` has to make in copy_src, copy_dst (int32, at least half as many as
    pages of the cache, -1 behind the copies), free_pages (int32 ``[pages of the cache]``) and num_free (int32 ``[1]``)."""
    workspace = _workspace(workspace, block_table, "block_table", stream)
    _done(_h._ext.compact_pages(block_table, seq_lens, page_size, new_table, copy_src, copy_dst, free_pages, num_free, workspace,
                                _raw(stream, block_table)), "kda_compact_pages")


def copy_pages(buffers, copy_src, copy_dst, *, workspace=None, stream=None):
    """``kda_copy_pages``: pages ``copy_src[i]`` -> ``copy_dst[i]`` (int32, a negative one: no copy) of every buffer: a list
    of tensors ``[pages, ...]`` of any types whose pages are contiguous, 16-byte aligned and a multiple of 16 bytes long:
    the keys and values of every layer, or pools of states and windows.  They may be slices of one tensor, but no page of one may
    meet a page of another."""
    if workspace is None:
        workspace = _workspace(None, copy_src, "copy_src", stream)
    _done(_h._ext.copy_pages(buffers, copy_src, copy_dst, workspace, _raw(stream, copy_src)), "kda_copy_pages")


def shared_prefix_workspace_size(B: int, T: int, Hq: int, Hk: int, num_groups: int) -> int:
    """Bytes of workspace ``shared_prefix_attention`` needs (whatever the lengths)."""
    return int(_b.load().kda_shared_prefix_workspace_size(*map(operator.index, (B, T, Hq, Hk, num_groups))))


def shared_prefix_attention(q, k_pages, v_pages, block_table, seq_lens, prefix_lens, group_starts, T=1, *, scale=None,
                            out=None, lse=None, workspace=None, stream=None):
    """``kda_shared_prefix_attention``: :func:`paged_attention` for batches whose requests share long prefixes, which are
    read once for all of a group.

    prefix_lens: int32 ``[groups]``, tokens that the requests of a group have in common (their contents; the whole pages
    among them are usually the same pages); group_starts: int32 ``[groups + 1]``, ascending: group g is the requests
    ``group_starts[g] .. group_starts[g + 1] - 1``.  The other arguments and the results as in :func:`paged_attention`."""
    if out is None or workspace is None:
        dev = _h._cuda(q, "q")
        if out is None:
            out = _h._rows_like(q, "q", stream)
        if workspace is None:
            workspace = _h._new_workspace(dev, stream, shared_prefix_workspace_size(
                seq_lens.numel(), T, q.shape[1], k_pages.shape[2], prefix_lens.numel()))
    _done(_h._ext.shared_prefix_attention(q, k_pages, v_pages, block_table, seq_lens, prefix_lens, group_starts, T, scale, out,
                                          lse, workspace, _raw(stream, q)), "kda_shared_prefix_attention")
    return out, lse
