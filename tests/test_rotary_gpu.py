"""Rotary positions with the store into the pages, against their 64-bit definition."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, i32, rotary_reference

pytestmark = pytest.mark.gpu

# The phase is rounded to fp32 once (2^-24 of at most half a turn: pi 2^-24 < 2^-22 in the angle), cos and sin by their
# functions and by mscale (2^-23 together), the products and their sum (2^-24 each): below 2^-21 of |a| + |b| in all.  Then the
# result is rounded to bf16, at most half a step: 2^-8 of it.
HALF, BEFORE = 2.0 ** -8, 2.0 ** -21


def close(got, ref, size):
    got = got.detach().double().cpu()
    bound = HALF * (ref.abs() + BEFORE * size) + BEFORE * size + 1e-38
    bad = (got - ref).abs() > bound
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / bound).max()))


def make(tokens, hq, hk, R, axes=1, page=16, far=1 << 20, padding=0, seed=0, fused=False, base=10000.0):
    g = torch.Generator().manual_seed(seed)
    rows = tokens + padding
    qkv = torch.randn((rows, hq + 2 * hk, D), generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(-far, far, (axes, rows), generator=g).to(torch.int32).cuda()
    w = (base ** (-torch.arange(R // 2) / (R // 2))).float().cuda()
    pages = -(-rows // page) * 2 + 1
    slots = torch.randperm(pages * page, generator=g)[:rows]
    slots[tokens:] = -1
    kp, vp = (torch.randn((pages, page, hk, D), generator=g).bfloat16().cuda() for _ in range(2))
    return q, k, v, pos, slots.cuda(), w, kp, vp


def check(q, k, v, pos, slots, w, kp, vp, axes=None, interleaved=False, mscale=1.0, out=None, status=0):
    page, total = kp.shape[1], kp.shape[0] * kp.shape[1]
    which = [0] * w.numel() if axes is None else list(axes)
    ok = ((slots >= 0) & (slots < total)).cpu()
    p2 = pos if pos.dim() == 2 else pos[None]
    q_ref = rotary_reference(q, p2, w, which, interleaved, mscale)
    k_ref = rotary_reference(k, p2, w, which, interleaved, mscale)
    keep_k, keep_v, v0 = kp.cpu().clone(), vp.cpu().clone(), v.cpu().clone()
    before = torch.full(q.shape, 5.0, dtype=torch.bfloat16) if out is None else out.cpu().clone()
    if out is None:
        out = before.cuda()
    ws = kda.make_workspace()
    got = kda.rotary_to_pages(q, k, v, pos, slots, w, kp, vp, axes=axes, interleaved=interleaved, mscale=mscale, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert got is out and kda.read_device_status(ws) == status
    close(out.cpu()[ok], q_ref[0][ok], q_ref[1][ok])
    assert torch.equal(out.cpu()[~ok], before[~ok])
    at = slots.cpu()[ok]
    close(kp.cpu()[at // page, at % page], k_ref[0][ok], k_ref[1][ok])
    assert torch.equal(vp.cpu()[at // page, at % page], v0[ok])
    for x, was in ((kp, keep_k), (vp, keep_v)):   # other rows of the cache
        x = x.cpu().clone()
        x[at // page, at % page] = was[at // page, at % page]
        assert torch.equal(x, was)
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,R,axes,page", [
    (1, 1, 1, 128, 1, 1), (1, 16, 2, 128, 1, 16), (3, 5, 1, 64, 2, 24), (64, 16, 2, 128, 1, 16), (17, 32, 8, 96, 3, 64),
    (200, 8, 8, 16, 4, 7), (1001, 4, 2, 32, 3, 256), (2500, 16, 2, 128, 3, 48), (130, 3, 3, 112, 2, 5), (9, 64, 1, 80, 1, 16)])
def test_rotary(tokens, hq, hk, R, axes, page, interleaved):
    x = make(tokens, hq, hk, R, axes, page, padding=tokens % 3, seed=tokens + R, fused=tokens % 2 == 0)
    check(*x, axes=[f * axes // (R // 2) for f in range(R // 2)], interleaved=interleaved)


def test_one_axis_is_a_row():
    x = list(make(40, 8, 2, 128))
    a = check(*x)
    x[3] = x[3][0]
    b = check(*x)
    assert torch.equal(a, b)


def test_interleaved_sections():
    # axes in turn (time, height, width, time, ...), as bytes and as numbers
    x = make(70, 8, 2, 128, axes=3, seed=3)
    axes = [f % 3 for f in range(64)]
    assert torch.equal(check(*x, axes=axes), check(*x, axes=bytes(axes)))


def test_far_positions_and_frequencies():
    # the largest positions; frequencies above one, of nothing, and the smallest
    x = list(make(256, 2, 1, 128, far=2 ** 31 - 1, seed=4))
    x[3][0, :4] = i32([2 ** 31 - 1, -2 ** 31, 0, -1])
    x[5][:8] = torch.tensor([0.0, 1e-30, 1e-42, 3.0, 100.5, 1.0, 0.3, -0.7], device="cuda")
    check(*x)


def test_frequencies_that_are_none():
    x = list(make(5, 2, 1, 64, seed=5))
    x[5][3], x[5][4], x[5][5] = float("nan"), float("inf"), 2.0 ** 24
    out = kda.rotary_to_pages(*x)
    for f in (3, 4, 5):
        assert torch.isnan(out[..., f]).all() and torch.isnan(out[..., f + 32]).all()
    assert torch.isfinite(out[..., :3]).all() and torch.isfinite(out[..., 64:]).all()


@pytest.mark.parametrize("mscale", [0.5, 1.2079, -1.0, 0.0])
def test_mscale(mscale):
    check(*make(33, 4, 2, 96, seed=6), mscale=mscale)


@pytest.mark.parametrize("fused", [False, True])
def test_in_place(fused):
    x = make(100, 8, 2, 128, padding=3, seed=7, fused=fused)
    check(*x, out=x[0])


def test_strided_pages():
    # keys and values of a page in one buffer; pages of heads
    for layout in range(2):
        q, k, v, pos, slots, w, kp, vp = make(50, 8, 2, 128, page=16, seed=8)
        if layout == 0:
            both = torch.zeros((kp.shape[0], 2, 16, 2, D), dtype=torch.bfloat16, device="cuda")
            kp, vp = both[:, 0], both[:, 1]
        else:
            kp, vp = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kp, vp))
        check(q, k, v, pos, slots, w, kp, vp)


def test_bad_slots_are_left_out():
    x = list(make(40, 4, 2, 128, seed=9))
    total = x[6].shape[0] * x[6].shape[1]
    for bad in (total, -2, 2 ** 40, -2 ** 40):
        x[4][11] = bad
        check(*x, status=kda.KDA_DEVICE_BAD_SLOT)
    x[4][11] = -1
    check(*x)


def test_no_tokens():
    x = make(0, 4, 2, 128)
    assert kda.rotary_to_pages(*x).shape == (0, 4, D)


def test_offsets_beyond_32_bits():
    pages, page, hk = 4200, 1024, 8
    kp = torch.empty((pages, page, hk, D), dtype=torch.bfloat16, device="cuda")
    assert kp.numel() > 2 ** 32
    vp = torch.empty_like(kp)
    q, k, v, pos, _, w, _, _ = make(5, 8, hk, 128, seed=10)
    slots = torch.tensor([pages * page - 1, 0, 4199 * 1024, 4100 * 1024 + 17, 5], device="cuda")
    kda.rotary_to_pages(q, k, v, pos, slots, w, kp, vp)
    ref, size = rotary_reference(k, pos, w, [0] * 64, False)
    close(kp.view(-1, hk, D)[slots], ref, size)
    assert torch.equal(vp.view(-1, hk, D)[slots], v)


def test_same_bits_in_a_graph_and_on_another_stream():
    q, k, v, pos, slots, w, kp, vp = make(90, 16, 2, 128, axes=3, seed=11)
    axes, ws = bytes(f % 3 for f in range(64)), kda.make_workspace()
    out = torch.zeros_like(q)
    call = lambda: kda.rotary_to_pages(q, k, v, pos, slots, w, kp, vp, axes=axes, out=out, workspace=ws)  # noqa: E731
    call()
    want = out.clone(), kp.clone(), vp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (out, kp, vp):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    page, at = kp.shape[1], slots
    assert torch.equal(kp[at // page, at % page], want[1][at // page, at % page])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kda.rotary_to_pages(q, k, v, pos, slots, w, kp, vp, axes=axes, stream=side)
    side.synchronize()
    assert torch.equal(other, want[0])
