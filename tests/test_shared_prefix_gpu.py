"""Attention over shared prefixes on the GPU against its 64-bit definition (every request alone)."""
import math
import random

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, i32
from hybrid_refs import paged_reference, rel_l2

pytestmark = pytest.mark.gpu

# As of the paged attention: a weight is rounded to bf16 before it meets its value and the output once more, two roundings
# of at most 2^-8 each (rel-L2 of a row's 128 channels); lse from fp32 scores and weights, below 1e-5 of it.
OUT_TOL = 2 * 2.0 ** -8
LSE_TOL = 2e-5


def make(groups, T, hq, hk, page, seed, alone=0, share_pages=True, std=1.5, width=None, spare=2):
    """groups: [(shared tokens, [own tokens of its requests])]; `alone` requests behind them.  Returns the call's arguments."""
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    rows, lens, starts, prefix, total = [], [], [0], [], 0
    copies = []   # (page to fill, page of the prefix, tokens)
    tails = [(p, t) for p, ts in groups for t in ts] + [(0, 40 + 30 * i) for i in range(alone)]
    for p, t in tails:
        total += -(-(p + t) // page)
    total += spare
    ids = list(range(total))
    r.shuffle(ids)
    at = 0
    for p, ts in groups:
        first = None
        for t in ts:
            n = -(-(p + t) // page)
            row = ids[at:at + n]
            at += n
            if first is None:
                first = row
            elif share_pages:
                row[:p // page] = first[:p // page]
            for c in range(-(-p // page)):
                if row[c] != first[c]:
                    copies.append((row[c], first[c], min(page, p - c * page)))
            rows.append(row)
            lens.append(p + t)
        starts.append(len(rows))
        prefix.append(p)
    for p, t in tails[len(rows):]:
        n = -(-t // page)
        rows.append(ids[at:at + n])
        at += n
        lens.append(t)
    k, v = (torch.randn((total, page, hk, D), generator=g).bfloat16() for _ in range(2))
    for a, b, n in copies:
        k[a, :n], v[a, :n] = k[b, :n], v[b, :n]
    # (a table as wide as a long context's, so that the call is not taken for one with next to nothing to share)
    tokens = (1 << 28) // (512 * hk * max(1, len(rows) - len(groups)))
    width = width or max([len(x) for x in rows] + [tokens // page + 1])
    table = torch.full((len(rows), width), -5, dtype=torch.int32)
    for b, x in enumerate(rows):
        table[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    table = table.cuda()
    q = (std * torch.randn((len(rows) * T, hq, D), generator=g)).bfloat16().cuda()
    return [q, k.cuda(), v.cuda(), table, i32(lens), i32(prefix), i32(starts)]


def run(x, T, scale=None, out=None):
    q, k = x[0], x[1]
    hq, hk = q.shape[1], k.shape[2]
    ws = torch.full((kda.shared_prefix_workspace_size(x[4].numel(), T, hq, hk, x[5].numel()),), 255, dtype=torch.uint8, device="cuda")
    ws[:1024] = 0
    lse = torch.full((q.shape[0], hq), 9.0, device="cuda")
    out, _ = kda.shared_prefix_attention(*x, T, scale=scale, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    return out, lse, kda.read_device_status(ws)


def check(x, T, scale=None, status=0, out=None, ref=None):
    out, lse, st = run(x, T, scale, out)
    assert st == status
    q, k, v, table, lens = x[:5]
    ref, ref_lse = ref or paged_reference(q, k, v, table, lens.tolist(), T, scale or D ** -0.5)
    worst = max(rel_l2(out[b], ref[b]) for b in range(q.shape[0]))
    assert worst <= OUT_TOL, worst
    fin = torch.isfinite(ref_lse)
    assert torch.equal(torch.isfinite(lse.cpu()), fin) and (lse.cpu()[~fin] == -math.inf).all()
    assert not fin.any() or float((lse.cpu()[fin] - ref_lse[fin]).abs().max()) <= LSE_TOL * (1 + float(ref_lse[fin].abs().max()))
    return out, lse


@pytest.mark.parametrize("groups,T,hq,hk,page", [
    ([(1, [1])], 1, 1, 1, 1), ([(100, [1, 1])], 1, 8, 1, 16), ([(128, [5, 70, 1])], 1, 16, 2, 16), ([(500, [40, 7, 1, 22])], 1, 16, 2, 16),
    ([(129, [3] * 17)], 1, 16, 2, 64), ([(700, [1 + 9 * i for i in range(33)])], 1, 8, 2, 24), ([(1000, [5] * 40)], 1, 12, 4, 256),
    ([(300, [4] * 70), (17, [9, 8]), (2000, [100])], 1, 16, 2, 16), ([(0, [50, 3]), (640, [1, 2, 3])], 1, 8, 2, 64),
    ([(257, [40, 6, 9])], 4, 16, 2, 16), ([(511, [8] * 9), (64, [8] * 2)], 8, 8, 1, 48), ([(90, [2, 3])], 2, 5, 1, 5),
    ([(400, [64, 70, 90])], 64, 2, 1, 32), ([(1500, [20] * 130)], 1, 4, 2, 1), ([(3000, [11] * 5)], 1, 40, 1, 64),
    ([(6000, [3] * 24)], 3, 16, 2, 128), ([(333, [1] * 300)], 1, 2, 2, 16)])
def test_shared_prefix(groups, T, hq, hk, page):
    check(make(groups, T, hq, hk, page, seed=len(groups) + T + page, alone=page % 3), T)


def test_the_same_as_paged_attention():
    x = make([(800, [30, 1, 200]), (77, [5] * 6)], 1, 16, 2, 16, seed=1, alone=2)
    out, lse = check(x, 1)
    l2 = torch.empty_like(lse)
    o2, _ = kda.paged_attention(*x[:5], 1, lse=l2)
    for b in range(out.shape[0]):
        assert rel_l2(out[b], o2[b]) <= 2 * OUT_TOL
    assert float((lse - l2).abs().max()) <= 2 * LSE_TOL * (1 + float(l2.abs().max()))


def test_pages_of_their_own():
    # the same contents in other pages
    check(make([(300, [5, 60, 9])], 1, 8, 2, 16, seed=2, share_pages=False), 1)


def test_narrow_table():
    check(make([(300, [5, 60, 9])], 1, 8, 2, 16, seed=3, width=30), 1)


def test_padding_requests():
    # lengths of 0 at the beginning of a group, within it, and of a whole group
    x = make([(200, [9, 8, 7, 6]), (100, [5, 5]), (300, [1])], 2, 8, 2, 16, seed=4)
    x[4][0] = x[4][2] = 0
    check(x, 2)
    x[4][4] = x[4][5] = 0
    check(x, 2)
    x[4][:] = 0
    check(x, 2)


def test_prefix_longer_than_what_is_seen():
    # a prefix that reaches into a request's new tokens, or is longer than it: what all new tokens see counts as shared
    x = make([(200, [3, 60])], 4, 8, 2, 16, seed=5)
    check(x, 4)
    x = make([(200, [3, 60]), (90, [8] * 3)], 2, 8, 2, 16, seed=6)
    x[4][0] = 130
    check(x, 2)
    x[4][0] = 1
    check(x, 2)
    x[5][1] = 5000
    x[5][0] = 16 * x[3].shape[1] + 7
    x[4][2:] = 95   # now their whole contents have to be the same
    for c in range(6):
        for b in (3, 4):
            for t in (x[1], x[2]):
                t[x[3][b, c].long()] = t[x[3][2, c].long()]
    check(x, 2)


def test_one_group_and_none():
    x = make([(64, [1] * 4)], 1, 8, 2, 16, seed=7, alone=3)
    check(x, 1)
    check(x[:5] + [i32([]), i32([0])], 1)
    q = torch.empty((0, 8, D), dtype=torch.bfloat16, device="cuda")
    assert kda.shared_prefix_attention(q, x[1], x[2], x[3][:0], x[4][:0], i32([]), i32([0]))[0].shape == (0, 8, D)


def test_requests_between_groups_attend_alone():
    x = make([(150, [9, 8]), (0, [70]), (260, [7, 40, 1])], 1, 8, 2, 16, seed=8, alone=2)
    x[5], x[6] = i32([260]), i32([3, 6])
    check(x, 1)


@pytest.mark.parametrize("starts", [[0, 3, 2], [0, 2, 99], [-1, 2, 5], [4, 2, 5], [5, 5, 4]])
def test_bad_groups(starts):
    x = make([(150, [9, 8]), (260, [7, 40, 1])], 1, 8, 2, 16, seed=9)
    x[6] = i32(starts)
    check(x, 1, status=kda.KDA_DEVICE_BAD_INDEX)


def test_bad_prefix_lengths():
    x = make([(150, [9, 8]), (260, [7, 40, 1])], 1, 8, 2, 16, seed=10)
    x[5] = i32([-1, 260])
    check(x, 1, status=kda.KDA_DEVICE_BAD_INDEX)


def test_bad_lengths_and_pages():
    x = make([(400, [9, 8, 7])], 1, 8, 2, 16, seed=11)
    q, k, v, table, lens = x[:5]
    for bad in (-1, 16 * table.shape[1] + 1):
        lens[1] = bad
        out, lse, status = run(x, 1)
        assert status == kda.KDA_DEVICE_BAD_COUNT
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        ref, _ = paged_reference(q, k, v, table, [409, 0, 407], 1)
        assert all(rel_l2(out[b], ref[b]) <= OUT_TOL for b in (0, 2))
    lens[1] = 408
    # a page of the prefix that is none: its tokens are left out for all that read the prefix
    table[:, 3] = k.shape[0]
    out, _, status = run(x, 1)
    assert status == kda.KDA_DEVICE_BAD_PAGE
    for b in range(3):
        n = 407 + 2 - b
        keep = [j for j in range(n) if j // 16 != 3]
        at = table[b].cpu().long()
        kk = torch.stack([k[at[j // 16], j % 16] for j in keep])[None]
        vv = torch.stack([v[at[j // 16], j % 16] for j in keep])[None]
        ref, _ = paged_reference(q[b:b + 1], kk, vv, torch.zeros((1, 1), dtype=torch.int32), [len(keep)], 1)
        assert rel_l2(out[b], ref[0]) <= OUT_TOL, b


@pytest.mark.parametrize("scale", [1.0, 0.01, -0.2])
def test_scales(scale):
    check(make([(300, [20, 6, 5])], 1, 8, 2, 16, seed=12, std=0.5), 1, scale=scale)


def test_scale_of_nothing():
    x = make([(300, [20, 6, 5])], 1, 8, 2, 16, seed=12)
    check(x, 1, scale=0.0, ref=paged_reference(*x[:4], x[4].tolist(), 1, 0.0))


def test_large_scores():
    # one token of the prefix takes nearly all the weight; the running maximum moves far between tiles
    x = make([(900, [7, 9, 60])], 1, 4, 1, 16, seed=13, std=6.0)
    q, k, table = x[0], x[1], x[3]
    for at in (5, 300, 650):
        k[int(table[0, at // 16]), at % 16] = q[0, :1] * (1 + at / 400)
    check(x, 1)


def test_scores_of_one_sign():
    # maxima far below zero
    x = make([(400, [7, 9])], 1, 4, 1, 16, seed=14)
    x[0][:] = 4.0
    x[1][:] = -x[1].abs() * 3
    check(x, 1)


@pytest.mark.parametrize("rise", [0.05, 0.5, 3.0, 40.0])
def test_scores_that_rise(rise):
    # from tile to tile by `rise`, downwards and upwards: maxima that follow never, at times and at every tile
    n = 1700
    for sign in (1, -1):
        x = make([(n, [9] * 5)], 1, 4, 1, 20, seed=19)
        q, k, v, table, lens = x[:5]
        q[:] = 1.0
        k *= 0.1
        at = torch.arange(n, device="cuda")
        level = sign * rise / 128 * (at - n / 2) / math.sqrt(D)   # (a key of c throughout: a score of c sqrt(128))
        for b in range(5):
            page = table[b, at // 20].long()
            k[page, at % 20] = (0.1 * torch.randn((n, 1, D), generator=torch.Generator().manual_seed(3)).cuda() + level[:, None, None]).bfloat16()
            v[page, at % 20] = v[table[0, at // 20].long(), at % 20]
        check(x, 1)


def test_prefix_that_begins_with_bad_pages():
    # tiles of nothing before the first tokens that count: for one page they are left out, for a prefix of them nothing is left
    x = make([(700, [9] * 3), (256, [4, 4])], 1, 4, 1, 64, seed=20)
    table, lens = x[3], x[4]
    table[:3, :5] = -1
    table[3:, :4] = x[1].shape[0]
    out, lse, status = run(x, 1)
    assert status == kda.KDA_DEVICE_BAD_PAGE
    for b, first in ((0, 5), (1, 5), (2, 5), (3, 4), (4, 4)):
        row = table[b:b + 1, first:].contiguous()
        ref, ref_lse = paged_reference(x[0][b:b + 1], x[1], x[2], row, [int(lens[b]) - 64 * first], 1)
        assert rel_l2(out[b], ref[0]) <= OUT_TOL
        assert float((lse[b].cpu() - ref_lse[0]).abs().max()) <= LSE_TOL * (1 + float(ref_lse.abs().max()))


@pytest.mark.parametrize("n", [200, 384, 500])
def test_what_is_not_seen_does_not_matter(n):
    # NaN and infinities in other pages, behind the requests' ends and in the rest of the prefix's last page
    x = make([(n, [33, 5, 70])], 2, 8, 2, 48, seed=15, share_pages=False)
    q, k, v, table, lens = x[:5]
    clean = check(x, 2)[0].clone()
    used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b, m in enumerate(lens.tolist()):
        for j in range(m):
            used[int(table[b, j // 48]), j % 48] = True
    k[~used.cuda()], v[~used.cuda()] = float("nan"), float("inf")
    assert torch.equal(check(x, 2)[0], clean)
    # own tokens of the group's first request lie behind the prefix, in its pages: they are only its own
    b0 = [int(table[0, n // 48]), n % 48]
    k[b0[0], b0[1]], v[b0[0], b0[1]] = float("nan"), float("-inf")
    out, _, _ = run(x, 2)
    assert torch.isnan(out[:2]).all()
    for b in range(2, 6):
        assert rel_l2(out[b], clean[b].cpu()) <= OUT_TOL


def test_nan_of_seen_tokens_is_kept():
    x = make([(600, [9] * 20)], 1, 8, 2, 16, seed=16)
    clean = check(x, 1)[0]
    k, table = x[1], x[3]
    k[int(table[0, 10]), 3, 1] = float("nan")
    out, _, _ = run(x, 1)
    assert torch.isnan(out[:, 4:]).all() and torch.equal(out[:, :4], clean[:, :4])
    k[int(table[0, 10]), 3, 1] = 0
    x[2][int(table[0, 10]), 3, 0, 5] = float("nan")
    out, _, _ = run(x, 1)
    assert torch.isnan(out[:, :4, 5]).all() and torch.isfinite(out[:, :4, :5]).all() and torch.isfinite(out[:, 4:]).all()


def test_infinite_scores():
    # a key of infinities: scores of plus and minus infinity as plain fp32 arithmetic has them (NaN where all weight is one's)
    x = make([(300, [9] * 3)], 1, 2, 1, 16, seed=17)
    q, k, table = x[0], x[1], x[3]
    q[:] = q.abs()
    k[int(table[0, 2]), 5] = float("-inf")
    ref = paged_reference(*x[:4], x[4].tolist(), 1)
    check(x, 1, ref=ref)


def test_strides():
    x = make([(500, [40, 7, 1, 22])], 1, 16, 2, 16, seed=18)
    q, k, v, table = x[:4]
    out, lse = check(x, 1)
    both = torch.empty((k.shape[0], 2, 16, 2, D), dtype=torch.bfloat16, device="cuda")
    both[:, 0], both[:, 1] = k, v
    heads = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v)]
    wide = torch.full((4, 16 * D + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :16 * D] = q.view(4, -1)
    room = torch.full((4, table.shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    room[:, :table.shape[1]] = table
    dst = torch.full((4, 16 * D + 8), 4.0, dtype=torch.bfloat16, device="cuda")
    for kk, vv in ((both[:, 0], both[:, 1]), heads):
        y = [wide[:, :16 * D].view(4, 16, D), kk, vv, room[:, :table.shape[1]], *x[4:]]
        o2, l2 = check(y, 1, out=dst[:, :16 * D].view(4, 16, D))
        assert torch.equal(out, o2) and torch.equal(lse, l2) and (dst[:, 16 * D:] == 4.0).all()


def test_offsets_beyond_32_bits():
    pages, page, hk = 4200, 1024, 8
    k = torch.empty((pages, page, hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        t[-4:].normal_(generator=g)
    q = torch.randn((3, 16, D), device="cuda", generator=g).bfloat16()
    order = [pages - 1, pages - 3, pages - 2]
    table = i32([order, order, order])
    lens = [2500, 2101, 2300]
    x = [q, k, v, table, i32(lens), i32([2100]), i32([0, 3])]
    small = torch.tensor([[3, 1, 2]] * 3, dtype=torch.int32)
    check(x, 1, ref=paged_reference(q, k[-4:], v[-4:], small, lens, 1))


def test_same_bits_again_and_in_a_graph():
    x = make([(2000, [30, 5, 9]), (100, [8] * 5)], 2, 16, 2, 16, seed=19, alone=1)
    hq, hk, T = 16, 2, 2
    ws = kda.make_workspace(nbytes=kda.shared_prefix_workspace_size(9, T, hq, hk, 2))
    out, lse = torch.empty_like(x[0]), torch.empty((18, hq), device="cuda")
    call = lambda: kda.shared_prefix_attention(*x, T, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    want = out.clone(), lse.clone()
    for _ in range(5):
        out.zero_()
        call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # other lengths and groups in the same buffers
    x[4].copy_(i32([2003, 2002, 0, 101, 105, 7, 3, 0, 2]))
    x[5].copy_(i32([1990, 90]))
    x[6].copy_(i32([0, 3, 5]))
    graph.replay()
    torch.cuda.synchronize()
    ref, _ = paged_reference(*x[:4], x[4].tolist(), T)
    assert max(rel_l2(out[b], ref[b]) for b in range(18)) <= OUT_TOL


def test_two_streams_with_workspaces_of_their_own():
    sets = [make([(3000 + 500 * i, [40, 1, 9, 7])], 1, 16, 2, 16, seed=20 + i) for i in range(2)]
    outs = [torch.zeros_like(s[0]) for s in sets]
    wss = [kda.make_workspace(nbytes=kda.shared_prefix_workspace_size(4, 1, 16, 2, 1)) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w, st in zip(sets, outs, wss, streams):
            kda.shared_prefix_attention(*s, 1, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        ref, _ = paged_reference(*s[:4], s[4].tolist(), 1)
        assert max(rel_l2(o[b], ref[b]) for b in range(4)) <= OUT_TOL


def test_outputs_that_the_call_allocates_are_the_given_streams():
    x = make([(300, [5, 60, 9])], 1, 8, 2, 16, seed=22)
    want = check(x, 1)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = kda.shared_prefix_attention(*x, 1, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = random.Random(seed)
    hk = r.choice([1, 2, 3])
    hq, T, page = hk * r.choice([1, 2, 4, 5, 8]), r.choice([1, 1, 2, 3, 5]), r.choice([1, 7, 16, 40, 64, 128])
    groups = [(r.choice([0, 1, r.randint(1, 300), r.randint(1, 2500)]), [r.randint(1, 150) for _ in range(r.choice([1, 2, 9, 40]))])
              for _ in range(r.randint(1, 5))]
    groups = [(p, [max(t, T) for t in ts]) for p, ts in groups]
    check(make(groups, T, hq, hk, page, seed=seed, alone=r.randint(0, 3)), T)
