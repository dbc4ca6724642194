"""Gated delta rule on the GPU against its 64-bit definition: prefill, verify, decode, and their use together."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from hybrid_refs import D, gdn_inputs, gdn_reference, rel_l2

pytestmark = pytest.mark.gpu

# Outputs are bf16: one rounding is at most 2^-8 of a value, so 2^-8 in rel-L2 at the most.  The recurrence runs in
# fp32: sums of 128 products and a few factors per step, each step's roundings (below 150 x 2^-24 of the state)
# contracted by the next ones.  The chunked form feeds the tensor cores with pairs of bf16 (a value's rounding is
# 2^-18 of it): six such roundings meet in a state, 6 x 2^-18 at the most; its outputs take one bf16 rounding of P,
# of U and of the result, 3 x 2^-8 at the most.
OUT_STEP = 2.0 ** -8
STATE_RECURRENT = 150 * 2.0 ** -24
STATE_CHUNKED = 6 * 2.0 ** -18


def _pool(slots, hv, seed):
    g = torch.Generator().manual_seed(seed)
    return (0.05 * torch.randn((slots, hv, D, D), generator=g)).cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prefill(x, lens, **kw):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return kda.gdn_chunk_prefill(*x, _i32(cu), torch.tensor(cu, dtype=torch.int32), **kw)


@pytest.mark.parametrize("lens,hk,hv", [
    ([1], 1, 1), ([2], 2, 2), ([63], 1, 2), ([64], 2, 2), ([65], 1, 4), ([128], 1, 1), ([200, 1, 0, 64, 130], 2, 4),
    ([0, 3], 1, 1), ([517], 3, 3), ([33] * 9, 5, 5)])
@pytest.mark.parametrize("initial", [False, True])
def test_prefill(lens, hk, hv, initial):
    x = gdn_inputs(sum(lens), hk, hv, seed=len(lens) + 100 * hv)
    pool = _pool(len(lens) + 2, hv, 7)
    slots = torch.arange(len(lens) + 1, 1, -1, dtype=torch.int32, device="cuda")[:len(lens)].contiguous()
    before = pool.clone()
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), hv))
    out, final = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=initial, workspace=ws)
    torch.cuda.synchronize()
    assert kda.read_device_status(ws) == 0
    assert torch.equal(pool, before)
    ref, _, ref_S = gdn_reference(x, lens, before[slots.long()] if initial else None)
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    for n in range(len(lens)):
        for h in range(hv):
            assert rel_l2(final[n, h], ref_S[n, h]) <= STATE_CHUNKED, (n, h)
    # and the final states into the pool, every other slot kept
    out2, none = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=initial, final_to_pool=True,
                          workspace=ws)
    assert none is None and torch.equal(out, out2)
    assert torch.equal(pool[slots.long()], final)
    rest = [i for i in range(pool.shape[0]) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("lens,hk,hv,a_mean", [
    ([64 * 16], 1, 1, -4.0), ([1537], 1, 1, -6.0), ([2048 + 63], 2, 4, -6.0), ([4033, 0, 130, 64, 1], 1, 2, -6.0),
    ([700, 3000, 2100], 2, 2, -4.0), ([2600], 1, 1, 3.0), ([2600], 1, 1, 3000.0), ([64 * 40], 4, 16, -8.0)])
def test_prefill_long_sequences(lens, hk, hv, a_mean):
    # few sequences, long enough to be cut into segments: the entering states come from products of 128 x 128 matrices,
    # whose pass and whose product add a rounding each per segment (16 at the most) to the state's; with |F| <= 1 and
    # |B| bounded as a state is, each is at most as large as a chunk pass's own
    x = gdn_inputs(sum(lens), hk, hv, seed=sum(lens), a_mean=a_mean)
    pool = _pool(len(lens) + 1, hv, 8)
    before = pool.clone()
    slots = torch.arange(len(lens), 0, -1, dtype=torch.int32, device="cuda")
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), hv))
    out, final = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=True, workspace=ws)
    out2, _ = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=True, final_to_pool=True, workspace=ws)
    torch.cuda.synchronize()
    assert kda.read_device_status(ws) == 0
    ref, _, ref_S = gdn_reference(x, lens, before[slots.long()], keep=False)
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    for n in range(len(lens)):
        for h in range(hv):
            assert rel_l2(final[n, h], ref_S[n, h]) <= STATE_CHUNKED, (n, h)
    assert torch.equal(out, out2) and torch.equal(pool[slots.long()], final) and torch.equal(pool[0], before[0])


def test_prefill_more_sequences_than_a_launch_takes():
    # 1024 sequences a launch; the second launch's long one is cut into segments
    g = torch.Generator().manual_seed(95)
    lens = torch.randint(0, 40, (1029,), generator=g).tolist() + [1500, 7]
    x = gdn_inputs(sum(lens), 1, 1, seed=96)
    pool = _pool(len(lens), 1, 97)
    before = pool.clone()
    slots = torch.randperm(len(lens), generator=g).to(torch.int32).cuda()
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), 1))
    out, none = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=True, final_to_pool=True, workspace=ws)
    assert none is None and kda.read_device_status(ws) == 0
    ref, _, ref_S = gdn_reference(x, lens, before[slots.long()], keep=False)
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    final = pool[slots.long()]
    for n in range(len(lens)):
        assert rel_l2(final[n], ref_S[n]) <= STATE_CHUNKED, n


def test_prefill_workspace_one_byte_short_is_refused():
    x = gdn_inputs(1600, 1, 2, seed=98)
    need = kda.gdn_prefill_workspace_size(1600, 1, 2)
    with pytest.raises(kda.KdaError):
        _prefill(x, [1600], workspace=kda.make_workspace(nbytes=need)[:need - 1])


@pytest.mark.parametrize("lens,hk,hv", [([13000], 8, 16), ([13000, 130], 5, 15), ([12800], 19, 38)])
def test_prefill_cut_against_pieces(lens, hk, hv):
    # long enough for half-way states; the same tokens in calls too short to be cut, the state handed on.  Either is
    # within the tolerances of the definition (the pieces' calls are compared with it above), so both together are within twice
    x = gdn_inputs(sum(lens), hk, hv, seed=61, a_mean=-7.0)
    pool = _pool(len(lens) + 1, hv, 62)
    slots = _i32(list(range(1, len(lens) + 1)))
    out, final = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=True)
    at = 0
    for n, length in enumerate(lens):
        for t in range(0, length, 900):
            some = slice(at + t, at + min(t + 900, length))
            part = [y[some] if y.shape[0] == sum(lens) else y for y in x]
            o, _ = _prefill(part, [part[0].shape[0]], state_pool=pool, slot_ids=slots[n:n + 1], load_initial=True, final_to_pool=True)
            assert rel_l2(out[some], o.cpu()) <= 2 * 3 * OUT_STEP
        at += length
        for h in range(hv):
            assert rel_l2(final[n, h], pool[n + 1, h].cpu()) <= 2 * STATE_CHUNKED, (n, h)


def test_prefill_long_sequence_keeps_channels_apart():
    # a NaN among one value channel's values of an early segment reaches that channel alone, from its 64-token chunk's
    # first token on (the chunk's tokens meet in one product, where 0 x NaN is NaN)
    x = gdn_inputs(2500, 1, 2, seed=21)
    clean, _ = _prefill(x, [2500])
    x[2][700, 1, 5] = float("nan")
    out, final = _prefill(x, [2500])
    assert torch.isnan(out[700:, 1, 5]).all() and torch.isnan(final[0, 1, :, 5]).all()
    out[640:, 1, 5] = clean[640:, 1, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("lens,hk,hv", [([10], 1, 2), ([11], 1, 2), ([3, 0, 10, 1], 2, 4), ([3, 0, 11, 1], 2, 4), ([8] * 30, 1, 1)])
@pytest.mark.parametrize("initial", [False, True])
def test_prefill_few_tokens(lens, hk, hv, initial):
    # around the length up to which a batch is taken token by token; a bad slot is skipped on either side
    x = gdn_inputs(sum(lens), hk, hv, seed=90)
    pool = _pool(len(lens) + 1, hv, 91)
    before = pool.clone()
    slots = torch.arange(len(lens), 0, -1, dtype=torch.int32, device="cuda")
    out, final = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=initial)
    ref, _, ref_S = gdn_reference(x, lens, before[slots.long()] if initial else None)
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    for n in range(len(lens)):
        assert rel_l2(final[n], ref_S[n]) <= STATE_CHUNKED
    slots[0] = -1
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), hv))
    _, none = _prefill(x, lens, state_pool=pool, slot_ids=slots, load_initial=initial, final_to_pool=True, workspace=ws)
    assert none is None and kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_SLOT
    assert torch.equal(pool[0], before[0]) and torch.equal(pool[len(lens)], before[len(lens)])
    for n in range(1, len(lens)):
        assert torch.equal(pool[int(slots[n])], final[n])


@pytest.mark.parametrize("a_mean", [-12.0, 3.0, 60.0, 3000.0])
def test_prefill_decays(a_mean):
    # from no decay at all to one that clears the state at every token; e^lambda underflows from about 60 on
    lens = [150, 70]
    x = gdn_inputs(sum(lens), 2, 2, seed=11, a_mean=a_mean)
    pool = _pool(2, 2, 3)
    out, final = _prefill(x, lens, state_pool=pool, slot_ids=_i32([1, 0]), load_initial=True)
    ref, _, ref_S = gdn_reference(x, lens, pool[[1, 0]])
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    assert rel_l2(final, ref_S) <= STATE_CHUNKED


@pytest.mark.parametrize("lens", [[150], [2100]])
@pytest.mark.parametrize("initial", [False, True])
def test_prefill_channels_of_any_size(lens, initial):
    # value channels from 10^-20 to 10^20, some of them growing on the way, some zero for a while: each is as accurate as
    # if it were alone
    x = gdn_inputs(sum(lens), 1, 2, seed=70, a_mean=-5.0)
    g = torch.Generator().manual_seed(71)
    size = (10.0 ** (40 * torch.rand((1, 2, D), generator=g) - 20)).cuda()
    size = size.repeat(sum(lens), 1, 1)
    size[40:, :, 3] *= 1e8
    size[100:, :, 4] *= 1e-8
    size[:90, :, 5] = 0.0
    x[2] = (x[2].float() * size).bfloat16()
    x[2][130:, :, 6] = 0.0
    pool = _pool(1, 2, 72) * size[0][None, :, None, :] if initial else None
    kw = dict(state_pool=pool.contiguous(), slot_ids=_i32([0]), load_initial=True) if initial else {}
    out, final = _prefill(x, lens, **kw)
    ref, _, ref_S = gdn_reference(x, lens, pool, keep=False)
    for h in range(2):
        for c in range(D):
            assert rel_l2(final[0, h, :, c], ref_S[0, h, :, c]) <= STATE_CHUNKED, (h, c)
            assert rel_l2(out[:, h, c], ref[:, h, c]) <= 3 * OUT_STEP, (h, c)


def test_prefill_keys_of_any_size_and_none():
    # keys from 10^-12 to 10^12 (the norm's 1e-6 counts for the small ones), queries likewise, some of them zero
    x = gdn_inputs(200, 1, 2, seed=73, a_mean=-5.0)
    g = torch.Generator().manual_seed(74)
    for i in (0, 1):
        x[i] = (x[i].float() * (10.0 ** (24 * torch.rand((200, 1, 1), generator=g) - 12)).cuda()).bfloat16()
        x[i][20 + i:200:7] = 0.0
    out, final = _prefill(x, [200])
    ref, _, ref_S = gdn_reference(x, [200])
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    assert rel_l2(final, ref_S) <= STATE_CHUNKED


def test_prefill_one_strong_decay_among_weak_ones():
    # a token that clears the state: pairs of tokens behind it keep their weak decays
    x = gdn_inputs(190, 1, 2, seed=12, a_mean=-2.0)
    x[3][20] = 500.0
    x[3][100] = 80.0
    out, final = _prefill(x, [190])
    ref, _, ref_S = gdn_reference(x, [190])
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    assert rel_l2(final, ref_S) <= STATE_CHUNKED


def test_prefill_equal_keys():
    # every key the same: the correction matrix is as far from the identity as it gets
    x = gdn_inputs(256, 1, 1, seed=13, a_mean=-6.0)
    x[1] = x[1][:1].expand(256, 1, D).contiguous()
    x[4].fill_(3.0)
    out, final = _prefill(x, [256])
    ref, _, ref_S = gdn_reference(x, [256])
    assert rel_l2(out, ref) <= 3 * OUT_STEP
    # Here the 64 corrections of a chunk cancel: S = k s^T with s' = e^b s + sum_i U_i, where sum_i U_i is of the size
    # of one value while the |U_i| add up to 64 of them, so a rounding is measured against that sum.  U = T R with
    # T_ii = beta, T_ij = -beta^2 (1 - beta)^(i - j - 1) e^(..) and e^(..) <= 1: the |T_ij| of a row add up to at most
    # 2 beta.  T's and R's roundings and the dropped product of their low parts are each at most 2^-18 of
    # sum_j |T_ij| |R_j| <= 2 beta max |R|, U's rounding 2^-18 of as much: 64 x 4 x 2 beta x 2^-18 x max |R| / |s|, with
    # |R_j| <= |v_j| + |s before|.  What earlier chunks leave in s enters only through R, whose sum of weights over a
    # chunk is below 1.
    beta = float(torch.sigmoid(x[4][0, 0].double()))
    v = x[2][:, 0].double().norm(dim=-1)
    s = ref_S[0, 0].norm()   # |k^| = 1
    bound = 64 * 4 * 2 * beta * 2.0 ** -18 * float((v[192:].max() + v.max()) / s)
    assert rel_l2(final, ref_S) <= bound


def test_prefill_in_place_from_a_fused_projection():
    hk, hv, lens = 2, 4, [100, 37]
    x = gdn_inputs(sum(lens), hk, hv, seed=14)
    fused = torch.full((sum(lens), (2 * hk + hv) * D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    gates = torch.full((sum(lens), 2 * hv + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    views = [fused[:, :hk * D].view(-1, hk, D), fused[:, hk * D:2 * hk * D].view(-1, hk, D),
             fused[:, 2 * hk * D:(2 * hk + hv) * D].view(-1, hv, D), gates[:, 1:1 + hv], gates[:, 1 + hv:1 + 2 * hv]]
    for view, src in zip(views, x):
        view.copy_(src)
    wide = torch.full((sum(lens), hv * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out, final = _prefill(views + x[5:], lens, out=wide[:, :hv * D].view(-1, hv, D))
    dense, final2 = _prefill(x, lens)
    assert torch.equal(out, dense) and torch.equal(final, final2)
    assert (wide[:, hv * D:] == 7.0).all()


def test_prefill_sequences_do_not_meet():
    # NaN and infinities in one sequence (and behind the last one) stay there
    lens = [70, 50, 90]
    x = gdn_inputs(sum(lens) + 30, 1, 2, seed=15)
    clean = [t[70:120].clone() if t.shape[0] == sum(lens) + 30 else t for t in x]
    for t in x[:5]:
        t[:70] = float("nan")
        t[120:] = float("inf")
    out, final = _prefill(x, lens)
    alone, final1 = _prefill(clean, [50])
    assert torch.equal(out[70:120], alone) and torch.equal(final[1], final1[0])
    assert torch.isnan(out[:70]).all() and torch.isnan(final[0]).all()


def test_prefill_bad_slot_is_skipped():
    lens = [20, 30]
    x = gdn_inputs(50, 1, 1, seed=16)
    pool = _pool(2, 1, 4)
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(50, 2, 1))
    out = torch.full((50, 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    final = torch.full((2, 1, D, D), 5.0, device="cuda")
    _prefill(x, lens, state_pool=pool, slot_ids=_i32([2, 1]), load_initial=True, out=out, final_state=final, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_SLOT
    assert (out[:20] == 5.0).all() and (final[0] == 5.0).all()
    ref, _, ref_S = gdn_reference([t[20:] if t.shape[0] == 50 else t for t in x], [30], pool[1:])
    assert rel_l2(out[20:], ref) <= 3 * OUT_STEP and rel_l2(final[1], ref_S[0]) <= STATE_CHUNKED


@pytest.mark.parametrize("B,T,hk,hv", [(1, 1, 1, 1), (3, 4, 2, 4), (2, 7, 3, 3), (1, 64, 1, 2), (5, 2, 1, 8)])
def test_verify(B, T, hk, hv):
    x = gdn_inputs(B * T, hk, hv, seed=B + 10 * T)
    pool = _pool(B + 1, hv, 5)
    before = pool.clone()
    slots = [(2 * b) % (B + 1) for b in range(B)]
    ws = kda.make_workspace()
    out, inter = kda.gdn_recurrent_verify(*x, pool, _i32(slots), T, workspace=ws)
    assert kda.read_device_status(ws) == 0 and torch.equal(pool, before)
    ref, steps, _ = gdn_reference(x, [T] * B, before[slots])
    assert rel_l2(out, ref) <= OUT_STEP
    for b in range(B):
        assert rel_l2(inter[b], steps[b]) <= STATE_RECURRENT


def test_verify_repeated_and_padding_slots():
    B, T, hv = 5, 3, 2
    x = gdn_inputs(B * T, 2, hv, seed=21)
    pool = _pool(3, hv, 6)
    ws = kda.make_workspace()
    out = torch.full((B * T, hv, D), 5.0, dtype=torch.bfloat16, device="cuda")
    inter = torch.full((B, T, hv, D, D), 5.0, device="cuda")
    kda.gdn_recurrent_verify(*x, pool, _i32([1, -1, 1, 7, 2]), T, out=out, intermediate_states=inter, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_SLOT   # of the 7 alone
    ref, steps, _ = gdn_reference(x, [T] * B, pool[[1, 0, 1, 0, 2]])
    for b in (0, 2, 4):
        assert rel_l2(out[b * T:(b + 1) * T], ref[b * T:(b + 1) * T]) <= OUT_STEP
        assert rel_l2(inter[b], steps[b]) <= STATE_RECURRENT
    for b in (1, 3):
        assert (out[b * T:(b + 1) * T] == 5.0).all() and (inter[b] == 5.0).all()


@pytest.mark.parametrize("B,hk,hv", [(1, 1, 1), (4, 2, 2), (7, 1, 4), (70, 8, 16)])
def test_decode(B, hk, hv):
    x = gdn_inputs(B, hk, hv, seed=30 + B)
    pool = _pool(B + 2, hv, 8)
    before = pool.clone()
    slots = list(range(B + 1, 1, -1))
    if B > 3:
        slots[2] = -1
    ws = kda.make_workspace()
    out = torch.full((B, hv, D), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.gdn_decode(*x, pool, _i32(slots), out=out, workspace=ws)
    assert kda.read_device_status(ws) == 0
    ref, _, ref_S = gdn_reference(x, [1] * B, before[slots])
    live = [b for b in range(B) if slots[b] >= 0]
    assert rel_l2(out[live], ref[live]) <= OUT_STEP
    assert rel_l2(pool[[slots[b] for b in live]], ref_S[live]) <= STATE_RECURRENT
    rest = [i for i in range(B + 2) if i not in slots]
    assert torch.equal(pool[rest], before[rest])
    if B > 3:
        assert (out[2] == 5.0).all()


def test_prefill_decode_verify_commit_together():
    """A prompt, two decoded tokens, a verified draft of which two tokens are accepted, and one more decoded token:
    the states and outputs are those of the whole sequence."""
    hk, hv, T = 1, 2, 4
    lens = [150, 65]
    total = [n + 2 + T + 1 for n in lens]
    x = gdn_inputs(sum(total), hk, hv, seed=40)
    first = [0, total[0]]

    def rows(lo, hi):
        idx = torch.cat([torch.arange(f + n + lo, f + n + hi) if lo >= 0 else torch.arange(f, f + n)
                         for f, n in zip(first, lens)]).cuda()
        return [t[idx] if t.shape[0] == sum(total) else t for t in x]

    pool = torch.zeros((4, hv, D, D), device="cuda")
    slots = _i32([3, 1])
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), 2, hv))
    outs = [_prefill(rows(-1, 0), lens, state_pool=pool, slot_ids=slots, final_to_pool=True, workspace=ws)[0]]
    for t in range(2):
        outs.append(kda.gdn_decode(*rows(t, t + 1), pool, slots, workspace=ws))
    vout, inter = kda.gdn_recurrent_verify(*rows(2, 2 + T), pool, slots, T, workspace=ws)
    kda.commit_accepted(pool, slots, _i32([2, 2]), inter, workspace=ws)
    after = [torch.arange(f + n + 4, f + n + 5) for f, n in zip(first, lens)]   # the token behind the accepted two
    nxt = [t[torch.cat(after).cuda()] if t.shape[0] == sum(total) else t for t in x]
    last = kda.gdn_decode(*nxt, pool, slots, workspace=ws)
    assert kda.read_device_status(ws) == 0
    ref, steps, _ = gdn_reference(x, total)
    for i, (f, n) in enumerate(zip(first, lens)):
        p0 = sum(lens[:i])
        assert rel_l2(outs[0][p0:p0 + n], ref[f:f + n]) <= 3 * OUT_STEP
        for t in range(2):
            assert rel_l2(outs[1 + t][i], ref[f + n + t]) <= 2 * OUT_STEP
        assert rel_l2(vout[i * T:(i + 1) * T], ref[f + n + 2:f + n + 2 + T]) <= 2 * OUT_STEP
        assert rel_l2(last[i], ref[f + n + 4]) <= 2 * OUT_STEP
        assert rel_l2(pool[int(slots[i])], steps[i][n + 4]) <= STATE_CHUNKED


def test_graph_replay_and_other_stream():
    lens, hv = [100, 30], 2
    x = gdn_inputs(sum(lens), 1, hv, seed=50)
    cu = [0, 100, 130]
    cu_d, cu_h = _i32(cu), torch.tensor(cu, dtype=torch.int32)
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(130, 2, hv))
    out = torch.zeros((130, hv, D), dtype=torch.bfloat16, device="cuda")
    final = torch.zeros((2, hv, D, D), device="cuda")
    pool, slots = _pool(4, hv, 9), _i32([2, 0])
    dec = [t[:2].clone() if t.shape[0] == 130 else t for t in x]
    dout = torch.zeros((2, hv, D), dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        kda.gdn_chunk_prefill(*x, cu_d, cu_h, out=out, final_state=final, workspace=ws, stream=stream)
        kda.gdn_decode(*dec, pool, slots, out=dout, workspace=ws, stream=stream)

    before = pool.clone()
    step()
    torch.cuda.synchronize()
    want = [out.clone(), final.clone(), dout.clone(), pool.clone()]
    pool.copy_(before)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()   # once outside the capture on its stream
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(2):
        for t in (out, final, dout):
            t.zero_()
        pool.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, final, dout, pool)))
    for t in (out, final, dout):
        t.zero_()
    pool.copy_(before)
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, final, dout, pool)))


@pytest.mark.parametrize("before", ["memset", "copy", "two streams", "kernel"])
def test_captured_behind_other_work(before):
    # the first launch of a call joins whatever the captured stream waits for: a memset, a copy, another stream's work
    hv, tokens = 2, 3
    x = gdn_inputs(tokens, 1, hv, seed=31)
    pool0 = _pool(4, hv, 9)
    pool, slots = torch.empty_like(pool0), _i32([2, 0, 3])
    long = gdn_inputs(130, 1, hv, seed=32)
    cu_h = torch.tensor([0, 100, 130], dtype=torch.int32)
    cu_d = cu_h.cuda()
    ws = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(130, 2, hv))
    ws2 = kda.make_workspace()
    out, out2 = torch.empty((tokens, hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((130, hv, D), dtype=torch.bfloat16, device="cuda")
    final = torch.empty((2, hv, D, D), device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        s = torch.cuda.current_stream()
        if before == "two streams":
            side.wait_stream(s)
            with torch.cuda.stream(side):
                pool.copy_(pool0)
            out.zero_()
            s.wait_stream(side)
        elif before == "kernel":
            torch.add(pool0, 0.0, out=pool)
        elif before == "memset":
            pool.copy_(pool0)
            out.view(torch.uint8).zero_()
        else:
            pool.copy_(pool0)
        kda.gdn_decode(*x, pool, slots, out=out, workspace=ws2)
        if before == "two streams":
            side.wait_stream(s)
            with torch.cuda.stream(side):
                out2.zero_()
            s.wait_stream(side)
        kda.gdn_chunk_prefill(*long, cu_d, cu_h, out=out2, final_state=final, workspace=ws)

    with torch.cuda.stream(main):
        work()
        torch.cuda.synchronize()
        want = [t.clone() for t in (pool, out, out2, final)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            work()
    for _ in range(3):
        for t in (pool, out, out2, final):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((pool, out, out2, final), want))


def test_two_streams_at_once():
    # prefills of different shapes (cut and whole), decodes beside them, each stream with its own workspace and pool
    shapes = [([300, 64, 500], 2, 4), ([2500], 1, 2)]
    runs = []
    for i, (lens, hk, hv) in enumerate(shapes):
        x = gdn_inputs(sum(lens), hk, hv, seed=80 + i, a_mean=-5.0)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        dec = [t[:3].contiguous() if t.shape[0] == sum(lens) else t for t in x]
        runs.append(dict(x=x, cu=_i32(cu), cu_h=torch.tensor(cu, dtype=torch.int32), dec=dec, pool=_pool(4, hv, 82 + i),
                         slots=_i32([3, 0, 1]), ws=kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), hv)),
                         out=torch.empty((sum(lens), hv, D), dtype=torch.bfloat16, device="cuda"),
                         final=torch.empty((len(lens), hv, D, D), device="cuda"),
                         dout=torch.empty((3, hv, D), dtype=torch.bfloat16, device="cuda")))

    def step(r, stream):
        kda.gdn_chunk_prefill(*r["x"], r["cu"], r["cu_h"], out=r["out"], final_state=r["final"], workspace=r["ws"], stream=stream)
        kda.gdn_decode(*r["dec"], r["pool"], r["slots"], out=r["dout"], workspace=r["ws"], stream=stream)

    want = []
    for r in runs:
        pool = r["pool"].clone()
        for _ in range(8):
            step(r, None)
        want.append([r[k].clone() for k in ("out", "final", "dout", "pool")])
        r["pool"].copy_(pool)
        for k in ("out", "final", "dout"):
            r[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for r, s in zip(runs, streams):
            step(r, s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert kda.read_device_status(r["ws"]) == 0
        assert all(torch.equal(a, r[k]) for a, k in zip(w, ("out", "final", "dout", "pool")))
