"""torch binding of the calls beside the KDA layers (``include/kda.h``): the gated delta rule, attention over a
paged key-value cache, and the step tables.

Tensors are checked for device, type, shape and strides before the library is called (``csrc/kda_torch.cpp``); a call
runs with the tensors' device current, on the given stream or that device's current one.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import operator
import os

import torch

from . import _binding as _b
from ._binding import KDA_FINAL_TO_POOL, KDA_LOAD_INITIAL, KDA_OK, KdaError

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


class _Unloaded:
    """Stands for the extension until the first call, which loads it and binds the library's entry points."""

    def __getattr__(self, name):
        global _ext
        from . import build

        lib = _b.load()
        path = build.torch_ext()
        if not os.path.exists(path):
            raise RuntimeError(f"the torch binding is not built for this interpreter and torch ({path} missing): run "
                               "__graft_entry__.build() or `python -m kda_linear_attention_bounded_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_kda_torch", path)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kda_torch", loader))
        loader.exec_module(ext)
        ext.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                   for f in ("kda_gdn_chunk_prefill", "kda_gdn_recurrent_verify", "kda_gdn_decode", "kda_paged_attention",
                             "kda_step_tables", "kda_rotary_to_pages", "kda_fork_requests", "kda_release_requests",
                             "kda_compact_pages", "kda_copy_pages", "kda_shared_prefix_attention")))
        _ext = ext
        return getattr(ext, name)


_ext = _Unloaded()


def _cuda(x, name):
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return x.device


def _raw(stream, x):
    """The stream's handle; it has to be one of x's device."""
    if stream.device != x.device:
        raise ValueError(f"stream: expected a stream of {x.device}")
    return stream.cuda_stream


def _rows_like(x, name, stream):
    """A new output for the tokens of x."""
    return _b._empty(x.shape, _BF16, _cuda(x, name), stream)


def _new_workspace(dev, stream, nbytes=None):
    with torch.cuda.device(dev):
        return _b.make_workspace(dev, stream, nbytes)


def gdn_prefill_workspace_size(total_tokens: int, num_seqs: int, Hv: int) -> int:
    """Bytes of workspace ``gdn_chunk_prefill`` needs."""
    return int(_b.load().kda_gdn_prefill_workspace_size(int(total_tokens), int(num_seqs), int(Hv)))


def gdn_chunk_prefill(q, k, v, a, beta_logits, A_log, dt_bias, cu_seqlens, cu_seqlens_host, *, scale=None,
                      state_pool=None, slot_ids=None, load_initial=False, final_to_pool=False, out=None,
                      final_state=None, workspace=None, stream=None):
    """``kda_gdn_chunk_prefill``: chunked varlen prefill of the gated delta rule.  q, k ``[tokens, Hk, 128]``, v
    ``[tokens, Hv, 128]``, a and beta_logits ``[tokens, Hv]`` (bf16), A_log and dt_bias ``[Hv]`` (fp32); the rest as
    in :func:`chunk_prefill`.  Returns ``(out, final_state)`` (final_state is None when the final states go to the
    pool)."""
    cu = cu_seqlens_host
    if cu.__class__ is not torch.Tensor or cu.dtype is not _I32 or not cu.is_contiguous():
        cu = torch.as_tensor(cu, dtype=_I32).contiguous()
    if out is None or workspace is None or (final_state is None and not final_to_pool):
        dev = _cuda(q, "q")
        N, Hv = max(cu.numel() - 1, 0), v.shape[1]
        if out is None:
            out = _rows_like(v, "v", stream)
        if final_state is None and not final_to_pool:
            final_state = _b._empty((N, Hv, 128, 128), _F32, dev, stream)
        if workspace is None:
            workspace = _new_workspace(dev, stream, gdn_prefill_workspace_size(q.shape[0], N, Hv))
    flags = (KDA_LOAD_INITIAL if load_initial else 0) | (KDA_FINAL_TO_POOL if final_to_pool else 0)
    rc = _ext.gdn_chunk_prefill(q, k, v, a, beta_logits, A_log, dt_bias, scale, cu_seqlens, cu, state_pool, slot_ids, flags,
                                out, final_state, workspace, None if stream is None else _raw(stream, q))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_chunk_prefill")
    return out, (None if final_to_pool else final_state)


def gdn_recurrent_verify(q, k, v, a, beta_logits, A_log, dt_bias, state_pool, slot_ids, T, *, scale=None, out=None,
                         intermediate_states=None, workspace=None, stream=None):
    """``kda_gdn_recurrent_verify``: T draft tokens per request from the pooled states, the state after every token
    recorded (``commit_accepted`` takes the records).  Returns ``(out, intermediate_states)``."""
    if out is None or intermediate_states is None or workspace is None:
        dev = _cuda(q, "q")
        if out is None:
            out = _rows_like(v, "v", stream)
        if intermediate_states is None:
            intermediate_states = _b._empty((slot_ids.numel(), max(operator.index(T), 0), v.shape[1], 128, 128), _F32, dev,
                                            stream)
        if workspace is None:
            workspace = _new_workspace(dev, stream)
    rc = _ext.gdn_recurrent_verify(q, k, v, a, beta_logits, A_log, dt_bias, scale, state_pool, slot_ids, T, out,
                                   intermediate_states, workspace, None if stream is None else _raw(stream, q))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_recurrent_verify")
    return out, intermediate_states


def gdn_decode(q, k, v, a, beta_logits, A_log, dt_bias, state_pool, slot_ids, *, scale=None, out=None,
               workspace=None, stream=None):
    """``kda_gdn_decode``: one token per request, its state updated in ``state_pool[slot_ids[b]]`` (distinct slots;
    rows of :data:`KDA_PAD_SLOT_ID` are skipped).  Returns ``out``."""
    if out is None or workspace is None:
        dev = _cuda(q, "q")
        if out is None:
            out = _rows_like(v, "v", stream)
        if workspace is None:
            workspace = _new_workspace(dev, stream)
    rc = _ext.gdn_decode(q, k, v, a, beta_logits, A_log, dt_bias, scale, state_pool, slot_ids, out, workspace,
                         None if stream is None else _raw(stream, q))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_decode")
    return out


def paged_workspace_size(Hq: int, Hk: int, T: int = 1) -> int:
    """Bytes of workspace ``paged_attention`` needs (whatever the batch and the lengths)."""
    return int(_b.load().kda_paged_workspace_size(*map(operator.index, (Hq, Hk, T))))


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, T=1, *, scale=None, out=None, lse=None,
                    workspace=None, stream=None):
    """``kda_paged_attention``: every request's T new tokens over its tokens in the paged cache.

    q: bf16 ``[B*T, Hq, 128]``; k_pages, v_pages: bf16 ``[pages, page_size, Hk, 128]`` with any page, token and head
    strides; block_table: int32 ``[B, width]``; seq_lens: int32 ``[B]``, the new tokens included (0: a padding row).
    lse: optional fp32 ``[B*T, Hq]`` to write.  Returns ``(out, lse)``."""
    if out is None or workspace is None:
        dev = _cuda(q, "q")
        if out is None:
            out = _rows_like(q, "q", stream)
        if workspace is None:
            workspace = _new_workspace(dev, stream, paged_workspace_size(q.shape[1], k_pages.shape[2], T))
    rc = _ext.paged_attention(q, k_pages, v_pages, block_table, seq_lens, T, scale, out, lse, workspace,
                              None if stream is None else _raw(stream, q))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_paged_attention")
    return out, lse


def step_tables(block_table, seq_lens, new_lens, free_pages, page_size, *, cu_seqlens, kv_lens, positions, slot_map,
                pages_used, workspace=None, stream=None):
    """``kda_step_tables``: page tables and slot maps of one step from the requests' lengths, all on the GPU.

    block_table: int32 ``[B, width]`` (rows may be strided), extended in place; seq_lens, new_lens: int32 ``[B]``;
    free_pages: int32 ``[F]``, taken from the front, negative ids behind the others not counted in.  Written: cu_seqlens int32 ``[B + 1]``, kv_lens int32 ``[B]``,
    positions int32 and slot_map int64 ``[rows]`` (padding rows: 0 and -1), pages_used int32 ``[1]``; none of them may overlap
    another or an input, but kv_lens may be seq_lens, which then moves forward in place."""
    if workspace is None:
        workspace = _new_workspace(_cuda(block_table, "block_table"), stream)
    rc = _ext.step_tables(block_table, seq_lens, new_lens, free_pages, page_size, cu_seqlens, kv_lens, positions, slot_map,
                          pages_used, workspace, None if stream is None else _raw(stream, block_table))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_step_tables")
