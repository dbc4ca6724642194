"""rotary_to_pages into keys and values that lie in one buffer, and on a cache of no pages."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, i32, rotary_reference

pytestmark = pytest.mark.gpu

P, T, H = 5, 8, 2


def views(name):
    """(the buffer, keys and values [P, T, H, D] in it)"""
    shape, pick = {
        "by page": ((P, 2, T, H, D), lambda x: (x[:, 0], x[:, 1])),
        "by token": ((P, T, 2, H, D), lambda x: (x[:, :, 0], x[:, :, 1])),
        "by head": ((P, T, H, 2, D), lambda x: (x[..., 0, :], x[..., 1, :])),
        "a layer of many": ((P, 3, 2, T, H, D), lambda x: (x[:, 1, 1], x[:, 1, 0])),
        "values heads first": ((P, 2, T * H, D), lambda x: (x[:, 0].view(P, T, H, D), x[:, 1].view(P, H, T, D).transpose(1, 2))),
        "heads outermost": ((2, H, P, T, D), lambda x: tuple(x[i].permute(1, 2, 0, 3) for i in range(2))),
    }[name]
    x = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    return x, *pick(x)


@pytest.mark.parametrize("name", ["by page", "by token", "by head", "a layer of many", "values heads first", "heads outermost"])
def test_keys_and_values_in_one_buffer(name):
    buffer, kp, vp = views(name)
    assert kp.shape == vp.shape == (P, T, H, D)
    g = torch.Generator().manual_seed(1)
    n = 23
    q, k, v = (torch.randn((n, h, D), generator=g).bfloat16().cuda() for h in (4, H, H))
    slots = torch.randperm(P * T, generator=g)[:n]
    pos = torch.randint(0, 9000, (n,), generator=g, dtype=torch.int32)
    freq = (10000.0 ** (-torch.arange(64) / 64)).float().cuda()
    kda.rotary_to_pages(q, k, v, pos.cuda(), slots.cuda(), freq, kp, vp)
    assert torch.equal(vp[slots // T, slots % T], v)
    want, size = rotary_reference(k, pos[None], freq, [0] * 64, False)
    # rounded once to bf16, cos and sin off by at most 2^-21
    assert ((kp[slots // T, slots % T].double().cpu() - want).abs() <= 2.0 ** -8 * (want.abs() + 2.0 ** -21 * size) + 2.0 ** -21 * size).all()
    for x in (kp, vp):
        x[slots // T, slots % T] = 7.0
    assert (buffer == 7).all()   # all else is as it was


def test_no_pages():
    """Keys and values of no pages may lie anywhere; the tokens' slots are none of theirs."""
    x = torch.zeros((4, T, H, D), dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.ones((3, h, D), dtype=torch.bfloat16, device="cuda") for h in (4, H, H))
    out, ws, freq = torch.full_like(q, 5.0), kda.make_workspace(), torch.ones(64, device="cuda")
    call = lambda pages, slots: kda.rotary_to_pages(q, k, v, i32([1, 2, 3]), torch.tensor(slots, device="cuda"), freq, pages, pages,  # noqa: E731
                                                    out=out, workspace=ws)
    call(x[:0], [-1, -1, -1])
    assert kda.read_device_status(ws) == 0 and (out == 5).all()
    call(x[:0], [-1, 0, 7])
    assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_SLOT and (out == 5).all() and (x == 0).all()
    with pytest.raises(kda.KdaError):
        call(x, [-1, 0, 7])
