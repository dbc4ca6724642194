"""Refusals of the calls beside the KDA layers, on the host (fake, aligned device addresses; never dereferenced) and
in the Python wrappers (CPU tensors)."""
import ctypes

import numpy as np
import pytest
import torch

from kda_linear_attention_bounded_gb300 import build as kbuild

FAKE = 0x10000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    from kda_linear_attention_bounded_gb300 import _binding
    return _binding.load()


def _head(hk=2, hv=4, q=FAKE, qs=None, v=FAKE, vs=None, a=FAKE, as_=None, beta=FAKE, A_log=FAKE, scale=0.1):
    return [P(q), P(FAKE), hk * 128 if qs is None else qs, P(v), hv * 128 if vs is None else vs, P(a),
            hv if as_ is None else as_, P(beta), hv, P(A_log), P(FAKE), scale], hk, hv


def _prefill(lib, *, cu=(0, 70), pool=None, slots=None, nslots=0, flags=0, out=FAKE, os_=None, final=FAKE, ws=FAKE,
             ws_bytes=None, **kw):
    head, hk, hv = _head(**kw)
    cu_host = np.array(cu, np.int32)
    if ws_bytes is None:
        ws_bytes = max(1024, lib.kda_gdn_prefill_workspace_size(max(int(cu[-1]), 0), len(cu) - 1, max(hv, 1)))
    return lib.kda_gdn_chunk_prefill(*head, P(FAKE), cu_host.ctypes.data_as(P), len(cu) - 1, hk, hv, P(pool), nslots,
                                     P(slots), flags, P(out), hv * 128 if os_ is None else os_, P(final), P(ws),
                                     ws_bytes, None)


BAD_TOKENS = [dict(hk=0), dict(hv=0), dict(hk=3), dict(hv=8192, hk=1), dict(q=None), dict(q=FAKE + 2),
              dict(v=None), dict(v=FAKE + 8), dict(a=None), dict(a=FAKE + 1), dict(beta=None), dict(A_log=None),
              dict(A_log=FAKE + 2), dict(qs=100), dict(qs=260), dict(qs=0), dict(vs=256), dict(vs=516), dict(as_=3)]


def test_gdn_prefill_refusals(lib):
    for bad in BAD_TOKENS:
        assert _prefill(lib, **bad) == 1, bad
    assert _prefill(lib, scale=float("nan")) == 2
    assert _prefill(lib, scale=float("inf")) == 2
    assert _prefill(lib, ws=None) == 3
    assert _prefill(lib, ws=FAKE + 64) == 3
    assert _prefill(lib, ws_bytes=1024 - 1) == 3
    assert _prefill(lib, cu=(0, 70, 60)) == 1
    assert _prefill(lib, cu=(2, 70)) == 1
    assert _prefill(lib, flags=4) == 1                 # the KDA calls' execution paths are not this call's
    assert _prefill(lib, flags=1) == 1                 # pool and slot ids required
    assert _prefill(lib, flags=2, pool=FAKE, slots=FAKE, nslots=0) == 1
    assert _prefill(lib, flags=2, pool=FAKE + 4, slots=FAKE, nslots=2) == 1
    assert _prefill(lib, final=None) == 1
    assert _prefill(lib, out=None) == 1
    assert _prefill(lib, os_=500) == 1
    assert _prefill(lib, cu=(0,)) == 0                 # no sequences: nothing to do


def _verify(lib, *, B=2, T=4, pool=FAKE, nslots=4, slots=FAKE, out=FAKE, inter=FAKE, ws=FAKE, ws_bytes=1024, **kw):
    head, hk, hv = _head(**kw)
    return lib.kda_gdn_recurrent_verify(*head, B, T, hk, hv, P(pool), nslots, P(slots), P(out), hv * 128, P(inter),
                                        P(ws), ws_bytes, None)


def _decode(lib, *, B=2, pool=FAKE, nslots=4, slots=FAKE, out=FAKE, ws=FAKE, ws_bytes=1024, **kw):
    head, hk, hv = _head(**kw)
    return lib.kda_gdn_decode(*head, B, hk, hv, P(pool), nslots, P(slots), P(out), hv * 128, P(ws), ws_bytes, None)


@pytest.mark.parametrize("call", [_verify, _decode])
def test_gdn_recurrent_refusals(lib, call):
    for bad in BAD_TOKENS:
        assert call(lib, **bad) == 1, bad
    assert call(lib, scale=float("nan")) == 2
    for bad in (dict(B=-1), dict(pool=None), dict(pool=FAKE + 4), dict(nslots=0), dict(slots=None), dict(out=None),
                dict(out=FAKE + 8)):
        assert call(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=512)):
        assert call(lib, **bad) == 3, bad
    assert call(lib, B=0) == 0
    if call is _verify:
        assert call(lib, T=0) == 1 and call(lib, T=65) == 1 and call(lib, inter=None) == 1


def _tables(lib, *, table=FAKE, stride=8, width=8, old=FAKE, new=FAKE, B=4, free=FAKE, num_free=5, page=16, rows=10,
            cu=FAKE, kv=FAKE, pos=FAKE, slot=FAKE, used=FAKE, ws=FAKE, ws_bytes=1024):
    return lib.kda_step_tables(P(table), stride, width, P(old), P(new), B, P(free), num_free, page, rows, P(cu), P(kv),
                               P(pos), P(slot), P(used), P(ws), ws_bytes, None)


def test_step_tables_refusals(lib):
    for bad in (dict(table=None), dict(stride=7), dict(old=None), dict(new=None), dict(B=-1), dict(free=None),
                dict(num_free=-1), dict(page=0), dict(page=-16), dict(rows=-1), dict(rows=2 ** 31), dict(cu=None),
                dict(kv=None), dict(pos=None), dict(slot=None), dict(used=None), dict(width=-1), dict(table=FAKE + 2),
                dict(slot=FAKE + 4), dict(cu=FAKE + 1)):
        assert _tables(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=512)):
        assert _tables(lib, **bad) == 3, bad


def test_wrappers_refuse_host_tensors(lib):
    import kda_linear_attention_bounded_gb300 as kda
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    g = torch.zeros((2, 1), dtype=torch.bfloat16)
    h = torch.zeros(1)
    pool, slots = torch.zeros((2, 1, 128, 128)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_decode(q, q, q, g, g, h, h, pool, slots)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_recurrent_verify(q, q, q, g, g, h, h, pool, slots, 1)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_chunk_prefill(q, q, q, g, g, h, h, slots, slots)
    z = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.step_tables(z[:2].view(1, 2), z[:1], z[:1], z, 16, cu_seqlens=z[:2], kv_lens=z[:1], positions=z,
                        slot_map=z.long(), pages_used=z[:1])


def test_wrappers_refuse_what_is_no_tensor(lib):
    import kda_linear_attention_bounded_gb300 as kda
    z = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="q: expected a tensor"):
        kda.gdn_decode(1, z, z, z, z, z, z, z, z, out=z, workspace=z)
    with pytest.raises(TypeError, match="block_table: expected a tensor"):
        kda.step_tables([[1]], z, z, z, 16, cu_seqlens=z, kv_lens=z, positions=z, slot_map=z, pages_used=z, workspace=z)
    with pytest.raises(ValueError, match="strided"):
        kda.gdn_decode(torch.eye(3).to_sparse(), z, z, z, z, z, z, z, z, out=z, workspace=z)


def _paged(lib, *, q=FAKE, qs=1024, k=FAKE, kps=4096, kts=256, khs=128, v=FAKE, vps=4096, num_pages=9, page=16,
           table=FAKE, ts=4, width=4, lens=FAKE, B=2, T=1, hq=8, hk=2, scale=0.1, out=FAKE, os_=1024, lse=None, ws=FAKE,
           ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = max(1024, lib.kda_paged_workspace_size(hq, hk, T))
    return lib.kda_paged_attention(P(q), qs, P(k), kps, kts, khs, P(v), vps, kts, khs, num_pages, page, P(table), ts, width,
                                   P(lens), B, T, hq, hk, scale, P(out), os_, P(lse), P(ws), ws_bytes, None)


def test_paged_refusals(lib):
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(qs=1016), dict(qs=1028), dict(k=None), dict(v=None),
                dict(k=FAKE + 4), dict(kps=-8), dict(kps=4), dict(kts=130), dict(khs=-128), dict(num_pages=-1),
                dict(page=0), dict(table=None), dict(table=FAKE + 2), dict(ts=3), dict(width=-1), dict(lens=None),
                dict(lens=FAKE + 2), dict(B=-1), dict(T=0), dict(T=65), dict(hk=0), dict(hk=3), dict(hq=0),
                dict(hq=8192), dict(out=None), dict(out=FAKE + 4), dict(os_=1000), dict(lse=FAKE + 2)):
        assert _paged(lib, **bad) == 1, bad
    assert _paged(lib, scale=float("nan")) == 2
    need = lib.kda_paged_workspace_size(8, 2, 1)
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert _paged(lib, **bad) == 3, bad
    assert _paged(lib, B=0) == 0
    assert lib.kda_paged_workspace_size(8, 3, 1) == 0 and lib.kda_paged_workspace_size(8, 2, 0) == 0


def test_paged_wrapper_refusals(lib):
    import kda_linear_attention_bounded_gb300 as kda
    with pytest.raises(ValueError, match="CUDA"):
        kda.paged_attention(torch.zeros((1, 2, 128), dtype=torch.bfloat16), None, None, None,
                            torch.zeros(1, dtype=torch.int32))
