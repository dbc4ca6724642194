"""Final states of the gated delta rule's prefill to the accuracy of an fp32 evaluation, whatever the inputs' sizes."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from gdn_rounding import final_states
from hybrid_refs import D, gdn_inputs, gdn_reference, rel_l2

# Outputs: a bf16 rounding of P, of U and of the result, 2^-8 each at most.
OUT = 3 * 2.0 ** -8
# A state is a sum of terms k^ u.  Besides S's own rounding a term carries eight relative errors of at most 2^-22 each: beta,
# the key's norm, the decay's two factors (approximate exponentials and reciprocal roots are good to 2^-22), L, R and U
# as pairs of fp16 (2^-23 each, with their products' sums 2^-22), and the sum of the terms.
TERM = 8 * 2.0 ** -22
# lengths and the mean of `a` (how weak the decays are): one chunk, a few, a ragged batch, long ones that are cut into segments
STATES = [([64], 0.0), ([200], 0.0), ([200], -6.0), ([64, 130, 11], -3.0), ([1100], -6.0)]


def state_bound(x, lens, S0=None):
    """Per sequence and head: the terms' errors and what S's rounding (two bf16) costs alone, both in rel-L2."""
    _, _, ref = gdn_reference(x, lens, S0, keep=False)
    got = final_states(x, lens, of_s=torch.bfloat16, S0=S0)
    return [[TERM + rel_l2(got[n, h], ref[n, h]) for h in range(ref.shape[1])] for n in range(len(lens))]


def _prefill(x, lens, **kw):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    cu = torch.tensor(cu, dtype=torch.int32)
    return kda.gdn_chunk_prefill(*x, cu.cuda(), cu, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,a_mean", STATES)
def test_states_are_an_fp32_evaluations(lens, a_mean):
    x = gdn_inputs(sum(lens), 2, 4, seed=len(lens) + sum(lens), a_mean=a_mean)
    out, final = _prefill(x, lens)
    ref, _, ref_S = gdn_reference(x, lens, keep=False)
    assert rel_l2(out, ref) <= OUT
    bound = state_bound(x, lens)
    for n in range(len(lens)):
        for h in range(4):
            assert rel_l2(final[n, h], ref_S[n, h]) <= bound[n][h], (n, h)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [2, 64])
def test_weak_decays_behind_a_strong_one(tokens):
    # A chunk's decays sum to 2^-45 or so after its first token, where an fp32 sum is good to 2^-19 and no more; the pairs
    # behind it differ by 2^-14 to 2^-3.  Equal keys and values, beta next to 1: a token's u is v minus what the state
    # holds already, so an error of A's entries is one of the state.
    # Two tokens: s = e^lambda u_0 + u_1 with u_1 = beta (v - e^lambda s_0), and s is v.  A's entry has two exponentials, the
    # first term one; beta and the norms (2^-23 each), the pairs of fp16 (2^-23 each) and the sums are not more than three
    # errors of 2^-22 besides.  Six errors of at most 2^-22 that do not know of each other have a root mean square of at most
    # (6 / 3)^(1/2) 2^-22 over many heads, below 2 x 2^-22.  With more tokens every u is such a difference, and they add up.
    hv = 64
    x = gdn_inputs(64, 1, hv, seed=5)
    for i in (0, 1, 2):
        x[i] = x[i][:1].expand_as(x[i])
    x[4].fill_(8.0)
    x[3][1:] = -3.0
    x[3][0] = (45 * 0.6931 / torch.exp(x[5]) - x[6]).bfloat16()
    x = [t[:tokens].contiguous() if i < 5 else t for i, t in enumerate(x)]
    # (padded by a sequence that is long enough for chunks)
    more = gdn_inputs(20, 1, hv, seed=6)
    x = [torch.cat([t, m]) if i < 5 else t for i, (t, m) in enumerate(zip(x, more))]
    out, final = _prefill(x, [tokens, 20])
    ref, _, ref_S = gdn_reference(x, [tokens, 20], keep=False)
    assert rel_l2(out, ref) <= OUT
    rms = (sum(rel_l2(final[0, h], ref_S[0, h]) ** 2 for h in range(hv)) / hv) ** 0.5
    assert rms <= tokens * 2.0 ** -22, rms


@pytest.mark.gpu
@pytest.mark.parametrize("initial", [False, True])
def test_values_next_to_the_largest_fade(initial):
    # a channel's value of 10^38 (or an entering state whose 1-norm passes fp32) decays by 2^-64 a chunk: four chunks later it
    # is nothing, and the channel is as accurate as any
    lens = [500]
    x = gdn_inputs(500, 1, 2, seed=6)
    x[3][:] = ((torch.log(torch.expm1(torch.tensor(0.6931, device="cuda") / torch.exp(x[5]))) - x[6])[None]).bfloat16()
    kw, S0 = {}, None
    if initial:
        S0 = torch.full((1, 2, D, D), 0.01, device="cuda")
        S0[..., 5] = 1e37
        kw = dict(state_pool=S0, slot_ids=torch.zeros(1, dtype=torch.int32, device="cuda"), load_initial=True)
    else:
        x[2][:20, :, 5] = 1e38
    out, final = _prefill(x, lens, **kw)
    ref, _, ref_S = gdn_reference(x, lens, S0, keep=False)
    for h in range(2):
        assert rel_l2(out[320:, h, 5], ref[320:, h, 5]) <= OUT
        assert rel_l2(final[0, h, :, 5], ref_S[0, h, :, 5]) <= TERM
        assert rel_l2(final[0, h], ref_S[0, h]) <= TERM


def _huge_rows(x, tokens):
    """Some keys and queries so long that their squares pass fp32 (and products with others, too)."""
    for i, (first, step) in ((0, (1, 5)), (1, (0, 4))):
        size = torch.ones((tokens, 1, 1), device="cuda")
        size[first::step] = 1e20
        size[first + 2::2 * step] = 1e30
        size[first + 3::3 * step] = 1e-18
        x[i] = (x[i].float() * size).bfloat16()
    x[1][2, 0] = 0.0
    x[1][2, 0, 7] = 3.3e38
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[200], [64], [9, 10], [9, 11], [70, 0, 3, 64, 1], [1100]])
@pytest.mark.parametrize("hk,hv", [(1, 2), (2, 2)])
def test_keys_whose_squares_pass_fp32(lens, hk, hv):
    x = _huge_rows(gdn_inputs(sum(lens), hk, hv, seed=8, a_mean=-4.0), sum(lens))
    out, final = _prefill(x, lens)
    ref, _, ref_S = gdn_reference(x, lens, keep=False)
    assert rel_l2(out, ref) <= OUT
    bound = state_bound(x, lens)
    for n in range(len(lens)):
        for h in range(hv):
            assert rel_l2(final[n, h], ref_S[n, h]) <= bound[n][h], (n, h)


@pytest.mark.gpu
def test_keys_whose_squares_pass_fp32_token_by_token():
    B, T, hv = 3, 4, 2
    x = _huge_rows(gdn_inputs(B * T, 1, hv, seed=9), B * T)
    g = torch.Generator().manual_seed(10)
    pool = (0.05 * torch.randn((B, hv, D, D), generator=g)).cuda()
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    out, inter = kda.gdn_recurrent_verify(*x, pool, slots, T)
    ref, steps, _ = gdn_reference(x, [T] * B, pool)
    assert rel_l2(out, ref) <= OUT
    for b in range(B):
        assert rel_l2(inter[b], steps[b]) <= 150 * 2.0 ** -24
    first = [t[::T].contiguous() if t.shape[0] == B * T else t for t in x]
    out1 = kda.gdn_decode(*first, pool, slots)
    assert torch.equal(out1, out[::T]) and torch.equal(pool, inter[:, 0])


@pytest.mark.gpu
def test_infinite_keys_still_spread():
    # an infinity among the keys is no number's norm: its chunk and what is behind it, in its own sequence, as it says
    lens = [100, 70]
    x = gdn_inputs(170, 1, 2, seed=11)
    clean = _prefill(x, lens)
    x[1][80, 0, 3] = float("inf")
    out, final = _prefill(x, lens)
    assert torch.equal(out[:64], clean[0][:64]) and torch.equal(out[100:], clean[0][100:])
    assert torch.isnan(out[80:100]).all() and torch.isnan(final[0]).all() and torch.equal(final[1], clean[1][1])
