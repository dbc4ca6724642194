"""Tensors that the calls beside the KDA layers refuse, argument by argument: another device, type, shape or layout.  Every
refusal is made on the host, so nothing is launched and nothing written."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from hybrid_refs import D, gdn_inputs

pytestmark = pytest.mark.gpu

HK, HV = 2, 4


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _gdn(tokens):
    return dict(zip(("q", "k", "v", "a", "beta_logits", "A_log", "dt_bias"), gdn_inputs(tokens, HK, HV, seed=1)))


def _prefill():
    cu = torch.tensor([0, 40, 60], dtype=torch.int32)
    return kda.gdn_chunk_prefill, dict(
        **_gdn(60), cu_seqlens=cu.cuda(), cu_seqlens_host=cu, state_pool=torch.zeros((4, HV, D, D), device="cuda"),
        slot_ids=_i32([1, 2]), load_initial=True, out=torch.zeros((60, HV, D), dtype=torch.bfloat16, device="cuda"),
        final_state=torch.zeros((2, HV, D, D), device="cuda"),
        workspace=kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(60, 2, HV)))


def _verify():
    return kda.gdn_recurrent_verify, dict(
        **_gdn(6), state_pool=torch.zeros((4, HV, D, D), device="cuda"), slot_ids=_i32([1, 2]), T=3,
        out=torch.zeros((6, HV, D), dtype=torch.bfloat16, device="cuda"),
        intermediate_states=torch.zeros((2, 3, HV, D, D), device="cuda"), workspace=kda.make_workspace())


def _decode():
    return kda.gdn_decode, dict(
        **_gdn(2), state_pool=torch.zeros((4, HV, D, D), device="cuda"), slot_ids=_i32([1, 2]),
        out=torch.zeros((2, HV, D), dtype=torch.bfloat16, device="cuda"), workspace=kda.make_workspace())


def _paged():
    pages = torch.zeros((2, 6, 16, HK, D), dtype=torch.bfloat16, device="cuda")
    return kda.paged_attention, dict(
        q=torch.zeros((4, HV, D), dtype=torch.bfloat16, device="cuda"), k_pages=pages[0], v_pages=pages[1],
        block_table=_i32([[0, 1, 2], [3, 4, 5]]), seq_lens=_i32([40, 3]), T=2,
        out=torch.zeros((4, HV, D), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((4, HV), device="cuda"),
        workspace=kda.make_workspace(nbytes=kda.paged_workspace_size(HV, HK, 2)))


def _tables():
    return kda.step_tables, dict(
        block_table=_i32([[0, 1, 2], [3, 4, 5]]), seq_lens=_i32([40, 3]), new_lens=_i32([1, 2]), free_pages=_i32([6, 7]),
        page_size=16, cu_seqlens=_i32([0] * 3), kv_lens=_i32([0] * 2), positions=_i32([0] * 5),
        slot_map=torch.zeros(5, dtype=torch.int64, device="cuda"), pages_used=_i32([0]), workspace=kda.make_workspace())


CALLS = {"prefill": _prefill, "verify": _verify, "decode": _decode, "paged": _paged, "tables": _tables}
# where fewer rows make another call that is right (fewer slots, fewer free pages)
FEWER = ("state_pool", "free_pages")


def _wider(t):
    """The same shape and values, its last dimension (and the rows' heads) further apart."""
    w = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=t.device)
    w[..., ::2] = t
    return w[..., ::2]


def _bad(name, t):
    yield "another device", t.cuda() if name == "cu_seqlens_host" else t.cpu()
    if name != "cu_seqlens_host":   # (host lengths are converted)
        yield "another type", t.to(torch.float16 if t.dtype is torch.bfloat16 else torch.float64 if t.is_floating_point()
                                   else torch.int16)
    yield "no tensor", 3
    if name != "workspace":   # (bytes of any shape)
        yield "a dimension more", t[None]
    if name not in FEWER and t.shape[0] > 1:
        yield "a row fewer", t[:-1]
    if t.shape[-1] > 1:
        yield "last dimension apart", _wider(t)
    if t.dim() > 1 and t.dtype is not torch.int32:
        yield "fewer in the last dimension", t[..., :-1].contiguous()


@pytest.mark.parametrize("name", CALLS)
def test_what_is_refused(name):
    call, args = CALLS[name]()
    call(**args)   # (as it should be)
    torch.cuda.synchronize()
    assert kda.read_device_status(args["workspace"]) == 0
    tensors = {k: t for k, t in args.items() if isinstance(t, torch.Tensor)}
    kept = {k: t.clone() for k, t in tensors.items()}
    for arg, t in tensors.items():
        for what, bad in _bad(arg, t):
            if arg == "cu_seqlens_host" and what == "last dimension apart":
                continue   # (host lengths are made contiguous)
            with pytest.raises((ValueError, TypeError, kda.KdaError)):
                call(**{**args, arg: bad})
                pytest.fail(f"{name}: {arg} of {what} was taken")
    torch.cuda.synchronize()
    for k, t in tensors.items():
        assert torch.equal(t, kept[k]), k


@pytest.mark.parametrize("name,arg", [("prefill", "q"), ("prefill", "v"), ("verify", "k"), ("decode", "v"), ("paged", "q"),
                                      ("prefill", "out"), ("paged", "out")])
def test_heads_apart_and_odd_places_are_refused(name, arg):
    call, args = CALLS[name]()
    t = args[arg]
    n, h, _ = t.shape
    apart = torch.zeros((n, 2 * h, D), dtype=t.dtype, device="cuda")[:, ::2]
    with pytest.raises(ValueError):
        call(**{**args, arg: apart})
    odd = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    with pytest.raises(kda.KdaError):
        call(**{**args, arg: odd})


def test_page_strides_that_are_refused():
    call, args = _paged()
    k = args["k_pages"]
    for shape, stride in (((6, 16, HK, D), (16 * 260, 260, 128, 1)), ((6, 16, HK, D), (16 * 256 + 4, 256, 128, 1))):
        room = torch.zeros(6 * 16 * 300, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(kda.KdaError):
            call(**{**args, "k_pages": room.as_strided(shape, stride)})
    with pytest.raises(ValueError, match="one shape"):
        call(**{**args, "k_pages": k[:5]})
    with pytest.raises(ValueError, match="overlap"):
        call(**{**args, "block_table": args["block_table"][:1].expand(2, 3)})


def test_lengths_that_are_refused():
    call, args = _prefill()
    for cu in ([0, 40, 61], [0, 40], [0, 50, 40], [1, 40, 60]):
        host = torch.tensor(cu, dtype=torch.int32)
        with pytest.raises((ValueError, kda.KdaError)):
            call(**{**args, "cu_seqlens_host": host})
    with pytest.raises(ValueError, match="slot_ids"):
        call(**{**args, "slot_ids": None})
    for name in ("verify", "paged"):
        f, a = CALLS[name]()
        for T in (0, -1, 4, 65):
            with pytest.raises((ValueError, kda.KdaError)):
                f(**{**a, "T": T})


def test_head_counts_that_are_refused():
    call, args = _decode()
    with pytest.raises(ValueError, match="multiple"):
        call(**{**args, "v": torch.zeros((2, 5, D), dtype=torch.bfloat16, device="cuda")})
    f, a = _paged()
    with pytest.raises(kda.KdaError):
        f(**{**a, **{k: torch.zeros((4, 3, D), dtype=torch.bfloat16, device="cuda") for k in ("q", "out")},
             "lse": torch.zeros((4, 3), device="cuda")})
