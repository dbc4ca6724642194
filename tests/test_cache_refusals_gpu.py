"""Tensors that the calls around the paged cache refuse, argument by argument: another device, type, shape or layout.  Every
refusal is made on the host, so nothing is launched and nothing written."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, i32
from test_refusals_gpu import _bad

pytestmark = pytest.mark.gpu

HK, HQ = 2, 4


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def _rotary():
    return kda.rotary_to_pages, dict(
        q=_bf16(6, HQ, D), k=_bf16(6, HK, D), v=_bf16(6, HK, D), positions=i32([[1] * 6, [2] * 6]),
        slot_map=torch.arange(6, device="cuda"), inv_freq=torch.ones(32, device="cuda"), k_pages=_bf16(4, 8, HK, D),
        v_pages=_bf16(4, 8, HK, D), out=_bf16(6, HQ, D), workspace=kda.make_workspace())


def _table():
    return i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]])


def _fork():
    return kda.fork_requests, dict(block_table=_table(), seq_lens=i32([20, 3, 0]), parents=i32([0, 1]), children=i32([2, 2]),
                                   free_pages=i32([9, 10]), page_size=16, copy_src=i32([0, 0]), copy_dst=i32([0, 0]),
                                   pages_used=i32([0]), workspace=kda.make_workspace())


def _release():
    return kda.release_requests, dict(block_table=_table(), seq_lens=i32([20, 3, 0]), rows=i32([1, 0]), page_size=16,
                                      free_pages=i32([0] * 12), num_free=i32([0]), workspace=kda.make_workspace())


def _compact():
    return kda.compact_pages, dict(block_table=_table(), seq_lens=i32([20, 3, 0]), page_size=16, new_table=_table(),
                                   copy_src=i32([0] * 6), copy_dst=i32([0] * 6), free_pages=i32([0] * 12), num_free=i32([0]),
                                   workspace=kda.make_workspace())


def _copy():
    return kda.copy_pages, dict(copy_src=i32([0, 1]), copy_dst=i32([2, 3]), workspace=kda.make_workspace())


def _prefix():
    return kda.shared_prefix_attention, dict(
        q=_bf16(6, HQ, D), k_pages=_bf16(9, 16, HK, D), v_pages=_bf16(9, 16, HK, D), block_table=_table(), seq_lens=i32([40, 33, 3]),
        prefix_lens=i32([32, 0]), group_starts=i32([0, 2, 3]), T=2, out=_bf16(6, HQ, D), lse=torch.zeros((6, HQ), device="cuda"),
        workspace=kda.make_workspace(nbytes=kda.shared_prefix_workspace_size(3, 2, HQ, HK, 2)))


CALLS = {"rotary": _rotary, "fork": _fork, "release": _release, "compact": _compact, "copy": _copy, "prefix": _prefix}
# what another size makes another call that is right (fewer frequencies, free pages, ended requests, a cache of fewer pages)
SIZES = ("free_pages", "rows", "inv_freq")


@pytest.mark.parametrize("name", CALLS)
def test_what_is_refused(name):
    call, args = CALLS[name]()
    extra = ([_bf16(9, 4, D)],) if name == "copy" else ()
    kept = {k: v.clone() for k, v in args.items() if isinstance(v, torch.Tensor)}
    tried = 0
    for arg, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        for why, bad in _bad(arg, t):
            if isinstance(bad, torch.Tensor) and arg in SIZES and why in ("a row fewer", "fewer in the last dimension"):
                continue
            if arg in ("k_pages", "v_pages") and why == "a row fewer":
                pass   # (pages of one shape only)
            if arg == "positions" and why in ("a row fewer",):
                continue   # one axis fewer
            if arg == "free_pages" and why == "a row fewer":
                continue
            with pytest.raises((ValueError, TypeError, kda.KdaError)):
                call(*extra, **{**args, arg: bad})
            tried += 1
    torch.cuda.synchronize()
    for k, v in kept.items():
        assert torch.equal(args[k], v), k
    assert tried >= 9


def test_buffers_that_are_refused():
    src, dst = i32([0]), i32([1])
    good = _bf16(9, 4, D)
    for bad in ([good, good[:8]], [good, good.cpu()], [good.transpose(1, 2)], [good[:, :, ::2]], [torch.zeros((9, 3), device="cuda")],
                [torch.zeros((9, 5), dtype=torch.uint8, device="cuda")[:, :4]], [good.expand(9, 4, D)[:, :1, :1]], [torch.zeros((), device="cuda")]):
        with pytest.raises((ValueError, kda.KdaError)):
            kda.copy_pages(bad, src, dst)


def test_frequencies_and_axes():
    call, args = _rotary()
    for half in (0, 4, 33, 72):
        with pytest.raises(kda.KdaError):
            call(**{**args, "inv_freq": torch.ones(half, device="cuda")})
    for axes in ([0] * 31, [2] * 32, b"\x00" * 33):
        with pytest.raises((ValueError, kda.KdaError)):
            call(**args, axes=axes)
    with pytest.raises(kda.KdaError):
        call(**args, mscale=float("inf"))
    call(**args, axes=[1] * 32)


def test_outputs_that_meet_inputs():
    call, args = _rotary()
    with pytest.raises(kda.KdaError):
        call(**{**args, "out": args["k_pages"].view(-1)[:6 * HQ * D].view(6, HQ, D)})
    with pytest.raises(kda.KdaError):   # a row behind q's own
        buf = _bf16(7, HQ, D)
        call(**{**args, "q": buf[:6], "out": buf[1:]})
    call, args = _fork()
    with pytest.raises(kda.KdaError):
        call(**{**args, "copy_src": args["copy_dst"]})
    call, args = _compact()
    with pytest.raises(kda.KdaError):
        call(**{**args, "num_free": args["free_pages"][3:4]})


def test_another_devices_stream():
    if torch.cuda.device_count() < 2:
        class Other:
            device, cuda_stream = torch.device("cuda", 1), 0
        stream = Other()
    else:
        stream = torch.cuda.Stream(device=1)
    for make in CALLS.values():
        call, args = make()
        with pytest.raises(ValueError, match="stream"):
            call(*(([_bf16(9, 4, D)],) if call is kda.copy_pages else ()), **args, stream=stream)
