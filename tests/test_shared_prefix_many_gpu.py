"""Attention over shared prefixes with more groups and more requests than the plan takes at once, against its 64-bit definition."""
import random

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import i32
from test_shared_prefix_gpu import check, make

pytestmark = pytest.mark.gpu


def many(groups, most, seed):
    r = random.Random(seed)
    return [(r.choice([0, 1, 8, r.randint(0, 90)]), [r.randint(1, 20) for _ in range(r.randint(1, most))]) for _ in range(groups)]


@pytest.mark.parametrize("groups,most,T,hq,hk", [(1023, 2, 1, 2, 1), (1024, 2, 1, 4, 2), (1025, 2, 1, 2, 2), (2300, 2, 1, 2, 1), (1100, 3, 2, 2, 1)])
def test_many_groups(groups, most, T, hq, hk):
    x = many(groups, most, groups)
    if T > 1:
        x = [(p, [n + T for n in ts]) for p, ts in x]
    check(make(x, T, hq, hk, 8, seed=groups, alone=3), T)


def test_many_requests_of_a_group():
    check(make([(70, [1 + i % 9 for i in range(1500)]), (33, [4] * 1100)], 1, 4, 1, 16, seed=5), 1)


def test_many_groups_with_requests_of_none():
    # padding requests in every window of groups, whole groups of them, requests before, between and behind the groups
    x = make(many(1400, 3, 6), 1, 2, 1, 8, seed=6, alone=40)
    q, k, v, table, lens, prefix, starts = x
    r = random.Random(7)
    for b in r.sample(range(lens.numel()), lens.numel() // 4):
        lens[b] = 0
    for g in (0, 700, 1030, 1399):
        lens[int(starts[g]):int(starts[g + 1])] = 0
    check(x, 1)
    x[5], x[6] = prefix[3:].contiguous(), starts[3:].contiguous()   # (the first requests are in no group)
    check(x, 1)


@pytest.mark.parametrize("g", [0, 1023, 1024, 1399])
def test_bad_bounds_behind_the_first_window(g):
    x = make(many(1400, 2, 8), 1, 2, 1, 8, seed=8)
    starts = x[6].tolist()
    starts[g + 1] = starts[g] - 1
    x[6] = i32(starts)
    check(x, 1, status=kda.KDA_DEVICE_BAD_INDEX)


def test_the_same_again():
    x = make(many(1500, 2, 9), 1, 2, 1, 8, seed=9)
    out, lse = check(x, 1)
    for _ in range(5):
        again, lse2 = kda.shared_prefix_attention(*x, 1, lse=torch.empty_like(lse))
        assert torch.equal(out, again) and torch.equal(lse, lse2)
