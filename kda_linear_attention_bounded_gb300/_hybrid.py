"""ctypes binding of the calls beside the KDA layers (``include/kda.h``): the gated delta rule, attention over a
paged key-value cache, and the step tables.

Argument marshalling only, as in ``_binding``.  Tensors are checked for device, type, shape and strides before the
library is called; a call runs with the tensors' device current, on the given stream or that device's current one.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as _b
from ._binding import KDA_FINAL_TO_POOL, KDA_LOAD_INITIAL, KDA_OK, KdaError

_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_SCALE = 128.0 ** -0.5
_no_guard = contextlib.nullcontext()


def _device_guard(dev):
    """A context in which ``dev`` is the current device (free when it is already)."""
    return _no_guard if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream: expected a stream of {dev}")
    return stream.cuda_stream


def _cuda(x, name):
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return x.device


def _check(x, name, dtype, dev, shape):
    """A contiguous CUDA tensor of this type, device and shape; returns its address."""
    if x.dtype != dtype or x.device != dev or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on {dev}, "
                         f"got {x.dtype} {list(x.shape)} on {x.device}")
    return x.data_ptr()


def _tokens(x, name, dev, tokens, H):
    """bf16 ``[tokens, H, 128]`` with contiguous heads; returns its token stride."""
    sh, st = x.shape, x.stride()
    if x.dtype != _BF16 or x.device != dev or len(sh) != 3 or sh[0] != tokens or sh[1] != H or sh[2] != 128 \
            or st[2] != 1 or (st[1] != 128 and H > 1):
        raise ValueError(f"{name}: expected a bf16 tensor [{tokens}, {H}, 128] on {dev} with contiguous heads")
    return st[0] if tokens > 1 else H * 128


def _scalars(x, name, dev, tokens, H):
    """bf16 ``[tokens, H]``; returns its token stride."""
    sh, st = x.shape, x.stride()
    if x.dtype != _BF16 or x.device != dev or len(sh) != 2 or sh[0] != tokens or sh[1] != H or (st[1] != 1 and H > 1):
        raise ValueError(f"{name}: expected a bf16 tensor [{tokens}, {H}] on {dev}, heads contiguous")
    return st[0] if tokens > 1 else H


def _workspace(ws, dev, stream, nbytes):
    if ws is None:
        return _b.make_workspace(dev, stream, nbytes)
    if ws.dtype != _U8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {dev}")
    return ws


def _pool(pool, name, dev, Hv):
    sh = pool.shape
    if pool.dtype != _F32 or pool.device != dev or len(sh) != 4 or sh[1] != Hv or sh[2] != 128 or sh[3] != 128 \
            or not pool.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous fp32 tensor [slots, {Hv}, 128, 128] on {dev}")
    return pool.data_ptr(), sh[0]


def _gdn_tokens(q, k, v, a, beta_logits, A_log, dt_bias, scale):
    """The common arguments of the gated-delta-rule calls: (device, tokens, Hk, Hv, C arguments)."""
    dev = _cuda(q, "q")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v: expected bf16 tensors [tokens, heads, 128]")
    tokens, Hk = q.shape[0], q.shape[1]
    Hv = v.shape[1]
    if Hk < 1 or Hv < 1 or Hv % Hk:
        raise ValueError(f"v: {Hv} value heads are not a multiple of q's and k's {Hk}")
    qs = _tokens(q, "q", dev, tokens, Hk)
    if _tokens(k, "k", dev, tokens, Hk) != qs:
        raise ValueError("q and k must share one token stride")
    args = (q.data_ptr(), k.data_ptr(), qs, v.data_ptr(), _tokens(v, "v", dev, tokens, Hv),
            a.data_ptr(), _scalars(a, "a", dev, tokens, Hv), beta_logits.data_ptr(),
            _scalars(beta_logits, "beta_logits", dev, tokens, Hv), _check(A_log, "A_log", _F32, dev, (Hv,)),
            _check(dt_bias, "dt_bias", _F32, dev, (Hv,)), _SCALE if scale is None else float(scale))
    return dev, tokens, Hk, Hv, args


def _out_rows(out, dev, tokens, H):
    if out is None:
        out = torch.empty((tokens, H, 128), dtype=_BF16, device=dev)
    return out, _tokens(out, "out", dev, tokens, H)


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
    lib = _b.load()
    dev, tokens, Hk, Hv, args = _gdn_tokens(q, k, v, a, beta_logits, A_log, dt_bias, scale)
    cu_host = torch.as_tensor(cu_seqlens_host, dtype=_I32).contiguous()
    if cu_host.is_cuda or cu_host.dim() != 1 or cu_host.numel() < 1:
        raise ValueError("cu_seqlens_host: expected host memory of [sequences + 1] entries")
    N = cu_host.numel() - 1
    if int(cu_host[-1]) > tokens:
        raise ValueError(f"cu_seqlens_host: its last entry {int(cu_host[-1])} lies behind the {tokens} tokens")
    cu = _check(cu_seqlens, "cu_seqlens", _I32, dev, (N + 1,))
    pool, slots, num_slots = None, None, 0
    if load_initial or final_to_pool:
        if state_pool is None or slot_ids is None:
            raise ValueError("load_initial and final_to_pool need state_pool and slot_ids")
        pool, num_slots = _pool(state_pool, "state_pool", dev, Hv)
        slots = _check(slot_ids, "slot_ids", _I32, dev, (N,))
    with _device_guard(dev):
        out, os_ = _out_rows(out, dev, tokens, Hv)
        final = None
        if not final_to_pool:
            if final_state is None:
                final_state = torch.empty((N, Hv, 128, 128), dtype=_F32, device=dev)
            final = _check(final_state, "final_state", _F32, dev, (N, Hv, 128, 128))
        if workspace is None:
            workspace = _b.make_workspace(dev, stream, gdn_prefill_workspace_size(tokens, N, Hv))
        else:
            _workspace(workspace, dev, stream, 0)
        flags = (KDA_LOAD_INITIAL if load_initial else 0) | (KDA_FINAL_TO_POOL if final_to_pool else 0)
        rc = lib.kda_gdn_chunk_prefill(*args, cu, cu_host.data_ptr(), N, Hk, Hv, pool, num_slots, slots, flags,
                                       out.data_ptr(), os_, final, workspace.data_ptr(), workspace.numel(),
                                       _stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_chunk_prefill")
    return out, (None if final_to_pool else final_state)


def gdn_recurrent_verify(q, k, v, a, beta_logits, A_log, dt_bias, state_pool, slot_ids, T, *, scale=None, out=None,
                         intermediate_states=None, workspace=None, stream=None):
    """``kda_gdn_recurrent_verify``: T draft tokens per request from the pooled states, the state after every token
    recorded (``commit_accepted`` takes the records).  Returns ``(out, intermediate_states)``."""
    lib = _b.load()
    dev, tokens, Hk, Hv, args = _gdn_tokens(q, k, v, a, beta_logits, A_log, dt_bias, scale)
    B, T = slot_ids.numel(), int(T)
    if tokens != B * T:
        raise ValueError(f"q: {tokens} tokens for {B} requests x {T}")
    pool, num_slots = _pool(state_pool, "state_pool", dev, Hv)
    slots = _check(slot_ids, "slot_ids", _I32, dev, (B,))
    with _device_guard(dev):
        out, os_ = _out_rows(out, dev, tokens, Hv)
        if intermediate_states is None:
            intermediate_states = torch.empty((B, T, Hv, 128, 128), dtype=_F32, device=dev)
        inter = _check(intermediate_states, "intermediate_states", _F32, dev, (B, T, Hv, 128, 128))
        workspace = _workspace(workspace, dev, stream, None)
        rc = lib.kda_gdn_recurrent_verify(*args, B, T, Hk, Hv, pool, num_slots, slots, out.data_ptr(), os_, inter,
                                          workspace.data_ptr(), workspace.numel(), _stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_recurrent_verify")
    return out, intermediate_states


def gdn_decode(q, k, v, a, beta_logits, A_log, dt_bias, state_pool, slot_ids, *, scale=None, out=None,
               workspace=None, stream=None):
    """``kda_gdn_decode``: one token per request, its state updated in ``state_pool[slot_ids[b]]`` (distinct slots;
    rows of :data:`KDA_PAD_SLOT_ID` are skipped).  Returns ``out``."""
    lib = _b.load()
    dev, tokens, Hk, Hv, args = _gdn_tokens(q, k, v, a, beta_logits, A_log, dt_bias, scale)
    pool, num_slots = _pool(state_pool, "state_pool", dev, Hv)
    slots = _check(slot_ids, "slot_ids", _I32, dev, (tokens,))
    with _device_guard(dev):
        out, os_ = _out_rows(out, dev, tokens, Hv)
        workspace = _workspace(workspace, dev, stream, None)
        rc = lib.kda_gdn_decode(*args, tokens, Hk, Hv, pool, num_slots, slots, out.data_ptr(), os_,
                                workspace.data_ptr(), workspace.numel(), _stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdn_decode")
    return out


def paged_workspace_size(Hq: int, Hk: int, T: int = 1) -> int:
    """Bytes of workspace ``paged_attention`` needs (whatever the batch and the lengths)."""
    return int(_b.load().kda_paged_workspace_size(int(Hq), int(Hk), int(T)))


def _pages(x, name, dev):
    """bf16 ``[pages, page_size, Hk, 128]``, channels contiguous; returns its shape and strides."""
    sh, st = x.shape, x.stride()
    if x.dtype != _BF16 or x.device != dev or len(sh) != 4 or sh[3] != 128 or st[3] != 1:
        raise ValueError(f"{name}: expected a bf16 tensor [pages, page_size, Hk, 128] on {dev}, channels contiguous")
    return sh, [0 if n == 1 else x for n, x in zip(sh, st)]


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, T=1, *, scale=None, out=None, lse=None,
                    workspace=None, stream=None):
    """``kda_paged_attention``: every request's T new tokens over its tokens in the paged cache.

    q: bf16 ``[B*T, Hq, 128]``; k_pages, v_pages: bf16 ``[pages, page_size, Hk, 128]`` with any page, token and head
    strides; block_table: int32 ``[B, width]``; seq_lens: int32 ``[B]``, the new tokens included (0: a padding row).
    lse: optional fp32 ``[B*T, Hq]`` to write.  Returns ``(out, lse)``."""
    lib = _b.load()
    dev = _cuda(q, "q")
    T = int(T)
    B = seq_lens.numel()
    if q.dim() != 3:
        raise ValueError("q: expected a bf16 tensor [B*T, Hq, 128]")
    Hq = q.shape[1]
    qs = _tokens(q, "q", dev, B * T, Hq)
    sh, ks = _pages(k_pages, "k_pages", dev)
    vsh, vs = _pages(v_pages, "v_pages", dev)
    if sh != vsh:
        raise ValueError("k_pages and v_pages must have one shape")
    if block_table.dtype != _I32 or block_table.device != dev or block_table.dim() != 2 or block_table.shape[0] != B or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table: expected an int32 tensor [{B}, width] on {dev} with contiguous rows")
    width = block_table.shape[1]
    lens = _check(seq_lens, "seq_lens", _I32, dev, (B,))
    lse_ptr = None if lse is None else _check(lse, "lse", _F32, dev, (B * T, Hq))
    with _device_guard(dev):
        out, os_ = _out_rows(out, dev, B * T, Hq)
        if workspace is None:
            workspace = _b.make_workspace(dev, stream, paged_workspace_size(Hq, sh[2], T))
        else:
            _workspace(workspace, dev, stream, 0)
        rc = lib.kda_paged_attention(
            q.data_ptr(), qs, k_pages.data_ptr(), ks[0], ks[1], ks[2], v_pages.data_ptr(), vs[0], vs[1], vs[2], sh[0],
            sh[1], block_table.data_ptr(), block_table.stride(0) if B > 1 else width, width, lens, B, T, Hq, sh[2],
            _SCALE if scale is None else float(scale), out.data_ptr(), os_, lse_ptr, workspace.data_ptr(),
            workspace.numel(), _stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_paged_attention")
    return out, lse


def step_tables(block_table, seq_lens, new_lens, free_pages, page_size, *, cu_seqlens, kv_lens, positions, slot_map,
                pages_used, workspace=None, stream=None):
    """``kda_step_tables``: page tables and slot maps of one step from the requests' lengths, all on the GPU.

    block_table: int32 ``[B, width]`` (rows may be strided), extended in place; seq_lens, new_lens: int32 ``[B]``;
    free_pages: int32 ``[F]``, taken from the front.  Written: cu_seqlens int32 ``[B + 1]``, kv_lens int32 ``[B]``,
    positions int32 and slot_map int64 ``[rows]`` (padding rows: 0 and -1), pages_used int32 ``[1]``."""
    lib = _b.load()
    dev = _cuda(block_table, "block_table")
    if block_table.dtype != _I32 or block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table: expected an int32 tensor [B, width] with contiguous rows")
    B, width = block_table.shape
    stride = block_table.stride(0) if B > 1 else width
    if stride < width:
        raise ValueError("block_table: its rows overlap")
    rows, free = slot_map.numel(), free_pages.numel()
    ptrs = (_check(cu_seqlens, "cu_seqlens", _I32, dev, (B + 1,)), _check(kv_lens, "kv_lens", _I32, dev, (B,)),
            _check(positions, "positions", _I32, dev, (rows,)), _check(slot_map, "slot_map", _I64, dev, (rows,)),
            _check(pages_used, "pages_used", _I32, dev, (1,)))
    with _device_guard(dev):
        workspace = _workspace(workspace, dev, stream, None)
        rc = lib.kda_step_tables(block_table.data_ptr(), stride, width, _check(seq_lens, "seq_lens", _I32, dev, (B,)),
                                 _check(new_lens, "new_lens", _I32, dev, (B,)), B,
                                 _check(free_pages, "free_pages", _I32, dev, (free,)), free, int(page_size), rows,
                                 *ptrs, workspace.data_ptr(), workspace.numel(), _stream(stream, dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_step_tables")
