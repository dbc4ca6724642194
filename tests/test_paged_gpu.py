"""Attention over a paged cache on the GPU against its 64-bit definition."""
import math

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from hybrid_refs import D, paged_reference, rel_l2

pytestmark = pytest.mark.gpu

# A weight is rounded to bf16 before it meets its value and the output once more: two roundings of at most 2^-8 each
# (rel-L2 of a row's 128 channels, where the weights' roundings meet as a sum of at most that much of each value's
# size; values here have one size).  Scores are sums of 128 products of bf16 in fp32 and e^x comes from ex2.approx
# (2^-22): below 1e-5 of l, so of lse in absolute terms.
OUT_TOL = 2 * 2.0 ** -8
LSE_TOL = 2e-5


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, T, hq, hk, page, seed, width=None, spare=2, std=1.5):
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + spare
    k = torch.randn((total, page, hk, D), generator=g).bfloat16().cuda()
    v = torch.randn((total, page, hk, D), generator=g).bfloat16().cuda()
    q = (std * torch.randn((len(lens) * T, hq, D), generator=g)).bfloat16().cuda()
    ids = torch.randperm(total, generator=g).tolist()
    width = width or max(pages + [1])
    table = torch.full((len(lens), width), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return q, k, v, table.cuda(), _i32(lens)


def check(q, k, v, table, lens, T, status=0, ref_lens=None, **kw):
    hq, hk = q.shape[1], k.shape[2]
    ws = torch.full((kda.paged_workspace_size(hq, hk, T),), 255, dtype=torch.uint8, device="cuda")
    ws[:1024] = 0
    lse = torch.full((q.shape[0], hq), 9.0, device="cuda")
    out, _ = kda.paged_attention(q, k, v, table, lens, T, lse=lse, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert kda.read_device_status(ws) == status
    scale = kw.get("scale") or D ** -0.5
    ref, ref_lse = paged_reference(q, k, v, table, lens.tolist() if ref_lens is None else ref_lens, T, scale)
    for b in range(q.shape[0]):
        assert rel_l2(out[b], ref[b]) <= OUT_TOL, b
    fin = torch.isfinite(ref_lse)
    assert torch.equal(torch.isfinite(lse.cpu()), fin)
    assert (lse.cpu()[~fin] == -math.inf).all()
    assert not fin.any() or float((lse.cpu()[fin] - ref_lse[fin]).abs().max()) <= LSE_TOL * (1 + float(ref_lse[fin].abs().max()))
    return out, lse


@pytest.mark.parametrize("lens,T,hq,hk,page", [
    ([1], 1, 1, 1, 1), ([1], 1, 8, 1, 16), ([63], 1, 16, 2, 16), ([64], 1, 4, 4, 64), ([65], 1, 16, 2, 24),
    ([257], 1, 16, 2, 16), ([1, 0, 700, 64, 3], 1, 8, 2, 16), ([2000, 5], 1, 5, 1, 5), ([300] * 9, 1, 12, 4, 256),
    ([40, 1000], 2, 16, 2, 16), ([4, 7, 900], 4, 8, 2, 64), ([66, 3], 8, 16, 2, 16), ([129], 3, 40, 1, 16),
    ([500, 64], 5, 16, 1, 1), ([33] * 40, 1, 16, 2, 16), ([1500, 2, 800], 64, 2, 1, 48), ([90, 200], 1, 17, 17, 8),
    ([20000], 1, 16, 2, 16), ([9000, 12, 4000, 700], 4, 32, 4, 64)])
def test_paged(lens, T, hq, hk, page):
    check(*make(lens, T, hq, hk, page, seed=len(lens) + T), T)


@pytest.mark.parametrize("lens,T,hq,hk,page", [
    ([1], 1, 16, 2, 16), ([0, 1, 64, 65], 1, 8, 2, 16), ([257], 1, 16, 2, 16), ([129, 2000], 1, 16, 2, 64),
    ([500, 3, 0, 1000, 64], 4, 8, 1, 16), ([1500], 8, 32, 4, 24), ([700, 20], 16, 8, 2, 5), ([130] * 40, 1, 16, 2, 16),
    ([90] * 160, 1, 8, 1, 64), ([2000, 1900], 2, 48, 2, 16), ([1, 2, 3], 3, 4, 4, 1)])
def test_clusters_and_stretches(lens, T, hq, hk, page):
    # a narrow table's items go to a cluster each, a wide one's (with no more tokens) are cut
    q, k, v, table, lens_d = make(lens, T, hq, hk, page, seed=len(lens) + 10 * T)
    out, lse = check(q, k, v, table, lens_d, T)
    wide = torch.full((len(lens), table.shape[1] + 40000 // page), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out2, lse2 = check(q, k, v, wide, lens_d, T)
    assert rel_l2(out2, out.cpu()) <= 2 * OUT_TOL or not out.any()
    # and the same bits again
    assert torch.equal(check(q, k, v, table, lens_d, T)[0], out) and torch.equal(check(q, k, v, wide, lens_d, T)[0], out2)


def test_more_requests_than_threads():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 90, (700,), generator=g).tolist()
    check(*make(lens, 1, 4, 2, 16, seed=4), 1)


def test_lengths_of_zero_only():
    check(*make([0, 0, 0], 1, 4, 2, 16, seed=5), 1)
    check(*make([0, 0], 3, 4, 2, 16, seed=5), 3)


def test_fewer_tokens_than_the_draft():
    # rows before the first token see nothing
    check(*make([2, 1, 0, 5], 4, 8, 2, 16, seed=6), 4)


@pytest.mark.parametrize("scale", [1.0, 0.01, -0.2])
def test_scales(scale):
    check(*make([300, 20], 1, 8, 2, 16, seed=7, std=0.5), 1, scale=scale)


def test_large_scores():
    # one token takes nearly all the weight; the running maximum moves far between tiles
    q, k, v, table, lens = make([400], 1, 4, 1, 16, seed=8, std=6.0)
    k[int(table[0, 20]), 3] = q[0, :1] * 2
    check(q, k, v, table, lens, 1)


def test_strides_and_interleaved_cache():
    q, k, v, table, lens = make([100, 333], 1, 8, 2, 16, seed=9)
    both = torch.empty((k.shape[0], 2, 16, 2, D), dtype=torch.bfloat16, device="cuda")   # K and V of a page together
    both[:, 0], both[:, 1] = k, v
    heads = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v)]              # pages of heads
    wide = torch.full((2, 8 * D + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :8 * D] = q.view(2, -1)
    out, lse = check(q, k, v, table, lens, 1)
    for kk, vv in ((both[:, 0], both[:, 1]), heads):
        o2, l2 = check(wide[:, :8 * D].view(2, 8, D), kk, vv, table, lens, 1)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    room = torch.full((2, table.shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    room[:, :table.shape[1]] = table
    o3, _ = check(q, k, v, room[:, :table.shape[1]], lens, 1)
    assert torch.equal(out, o3)
    dst = torch.full((2, 8 * D + 8), 4.0, dtype=torch.bfloat16, device="cuda")
    check(q, k, v, table, lens, 1, out=dst[:, :8 * D].view(2, 8, D))
    assert (dst[:, 8 * D:] == 4.0).all()


@pytest.mark.parametrize("width", [None, 4000])
def test_what_is_not_seen_does_not_matter(width):
    # NaN and infinities in other pages, behind the last token of the last page, and in later new tokens
    q, k, v, table, lens = make([70, 131], 3, 8, 2, 16, seed=10, width=width)
    clean = check(q, k, v, table, lens, 3)[0].clone()
    used = torch.zeros((k.shape[0], 16), dtype=torch.bool)
    for b, n in enumerate([70, 131]):
        for j in range(n):
            used[int(table[b, j // 16]), j % 16] = True
    k[~used.cuda()], v[~used.cuda()] = float("nan"), float("inf")
    assert torch.equal(check(q, k, v, table, lens, 3)[0], clean)
    for b, n in enumerate([70, 131]):
        last = int(table[b, (n - 1) // 16]), (n - 1) % 16
        k[last], v[last] = float("nan"), float("-inf")
    ws = kda.make_workspace(nbytes=kda.paged_workspace_size(8, 2, 3))
    out, _ = kda.paged_attention(q, k, v, table, lens, 3, workspace=ws)
    for b in range(2):
        assert rel_l2(out[b * 3], clean[b * 3].cpu()) <= OUT_TOL
        assert rel_l2(out[b * 3 + 1], clean[b * 3 + 1].cpu()) <= OUT_TOL
        assert torch.isnan(out[b * 3 + 2]).all()


@pytest.mark.parametrize("width", [None, 4000])
@pytest.mark.parametrize("tile", [0, 2, 6])
def test_nan_of_seen_tokens_is_kept(tile, width):
    # also where it is all that one CTA of an item sees
    q, k, v, table, lens = make([500, 130], 1, 8, 2, 16, seed=14, width=width)
    clean = check(q, k, v, table, lens, 1)[0]
    for j in range(64 * tile, min(64 * tile + 64, 500)):
        k[int(table[0, j // 16]), j % 16, 1] = float("nan")
    out, _ = kda.paged_attention(q, k, v, table, lens, 1)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.equal(out[0, :4], clean[0, :4]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("bad", [0, 1, 77, 149, 399])
@pytest.mark.parametrize("longest", [40, 700])
def test_a_bad_length_is_recorded_wherever_it_is(bad, longest):
    # with items cut and whole, whichever CTA has it
    B = 150 if bad < 150 else 400
    q, k, v, table, lens = make([1 + 37 * i % longest for i in range(B)], 1, 8, 1, 16, seed=12)
    good, _ = check(q, k, v, table, lens, 1)
    for n in (-1, 16 * table.shape[1] + 1):
        wrong = lens.clone()
        wrong[bad] = n
        ws = kda.make_workspace(nbytes=kda.paged_workspace_size(8, 1, 1))
        out, _ = kda.paged_attention(q, k, v, table, wrong, 1, workspace=ws)
        assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_COUNT
        assert (out[bad] == 0).all()
        rest = [b for b in range(B) if b != bad]
        assert rel_l2(out[rest], good[rest].cpu()) <= 2 * OUT_TOL


@pytest.mark.parametrize("hk,page,pages", [(1, 16, 30), (1, 64, 30), (3, 512, 1), (1, 512, 1)])
def test_strides_of_one_head_or_page_do_not_matter(hk, page, pages):
    q, k, v, table, lens = make([page * pages - 3], 1, 4 * hk, hk, page, seed=13, spare=0)
    out, _ = check(q, k, v, table, lens, 1)
    st = [0 if n == 1 else s for n, s in zip(k.shape, k.stride())]
    k0, v0 = (t.as_strided(t.shape, st) for t in (k, v))
    assert torch.equal(check(q, k0, v0, table, lens, 1)[0], out)


@pytest.mark.parametrize("width", [None, 4000])
def test_bad_pages_and_lengths_are_left_out(width):
    q, k, v, table, lens = make([100, 200, 50], 1, 8, 2, 16, seed=11, width=width)
    table[1, 4], table[1, 7] = k.shape[0], -1
    lens[2] = 16 * table.shape[1] + 1
    ws = kda.make_workspace(nbytes=kda.paged_workspace_size(8, 2, 1))
    lse = torch.zeros((3, 8), device="cuda")
    out, _ = kda.paged_attention(q, k, v, table, lens, 1, lse=lse, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_PAGE | kda.KDA_DEVICE_BAD_COUNT
    keep = [j for j in range(200) if j // 16 not in (4, 7)]
    at = table[1].cpu().long()
    kk = torch.stack([k[at[j // 16], j % 16] for j in keep])[None]
    vv = torch.stack([v[at[j // 16], j % 16] for j in keep])[None]
    ref, _ = paged_reference(q[1:2], kk, vv, torch.zeros((1, 1), dtype=torch.int32), [len(keep)], 1)
    assert rel_l2(out[1], ref[0]) <= OUT_TOL
    assert rel_l2(out[0], paged_reference(q[:1], k, v, table[:1], [100], 1)[0][0]) <= OUT_TOL
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_offsets_beyond_32_bits():
    # a cache of 2^32 + elements per tensor, only its last pages in use
    pages, page, hk = 4200, 1024, 8
    k = torch.empty((pages, page, hk, D), dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 32
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        t[-3:].normal_(generator=g)
    q = torch.randn((1, 8, D), device="cuda", generator=g).bfloat16()
    table = _i32([[pages - 1, pages - 3, pages - 2]])
    ws = kda.make_workspace(nbytes=kda.paged_workspace_size(8, hk, 1))
    out, _ = kda.paged_attention(q, k, v, table, _i32([2500]), workspace=ws)
    ref, _ = paged_reference(q, k[-3:], v[-3:], _i32([[2, 0, 1]]), [2500], 1)
    assert kda.read_device_status(ws) == 0 and rel_l2(out[0], ref[0]) <= OUT_TOL


def test_same_bits_again_and_in_a_graph():
    q, k, v, table, lens = make([5000, 30, 900, 0], 2, 16, 2, 16, seed=12)
    ws = kda.make_workspace(nbytes=kda.paged_workspace_size(16, 2, 2))
    out, lse = torch.empty_like(q), torch.empty((8, 16), device="cuda")
    call = lambda: kda.paged_attention(q, k, v, table, lens, 2, out=out, lse=lse, workspace=ws)  # noqa: E731
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
    # other lengths in the same buffers, as a captured bucket is replayed
    lens.copy_(_i32([7, 29, 0, 0]))
    graph.replay()
    torch.cuda.synchronize()
    ref, _ = paged_reference(q, k, v, table, [7, 29, 0, 0], 2)
    for b in range(8):
        assert rel_l2(out[b], ref[b]) <= OUT_TOL


def test_two_streams_with_workspaces_of_their_own():
    sets = [make([3000 + 500 * i, 40], 1, 16, 2, 16, seed=20 + i) for i in range(2)]
    outs = [torch.zeros_like(s[0]) for s in sets]
    wss = [kda.make_workspace(nbytes=kda.paged_workspace_size(16, 2, 1)) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w, st in zip(sets, outs, wss, streams):
            kda.paged_attention(*s, 1, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        ref, _ = paged_reference(*s[:4], s[4].tolist(), 1)
        for b in range(2):
            assert rel_l2(o[b], ref[b]) <= OUT_TOL


def test_step_tables_then_attention():
    """A prompt and then decoded tokens of three requests, through the step tables, the cache and the attention: as a
    user's decode loop calls them."""
    hq, hk, page, B, width = 8, 2, 16, 3, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    total = 40
    cache = torch.zeros((2, total, page, hk, D), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    cached = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = [[[], []] for _ in range(B)]
    ws = kda.make_workspace(nbytes=kda.paged_workspace_size(hq, hk, 1))
    for new in ([17, 0, 45], [1, 1, 1], [1, 30, 0], [1, 1, 1]):
        rows = 96
        outs = dict(cu_seqlens=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                    kv_lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
                    positions=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                    slot_map=torch.zeros(rows, dtype=torch.int64, device="cuda"),
                    pages_used=torch.zeros(1, dtype=torch.int32, device="cuda"))
        kda.step_tables(table, cached, _i32(new), free, page, workspace=ws, **outs)
        kv = torch.randn((2, rows, hk, D), generator=g, device="cuda").bfloat16()
        live = outs["slot_map"] >= 0
        for i in range(2):
            cache[i].view(-1, hk, D)[outs["slot_map"][live]] = kv[i][live]
        cu = outs["cu_seqlens"].tolist()
        for b in range(B):
            for i in range(2):
                history[b][i].append(kv[i, cu[b]:cu[b + 1]])
        q = torch.randn((B, hq, D), generator=g, device="cuda").bfloat16()
        out, _ = kda.paged_attention(q, cache[0], cache[1], table, outs["kv_lens"], workspace=ws)
        for b in range(B):
            k, v = (torch.cat(h)[None] for h in history[b])
            ref, _ = paged_reference(q[b:b + 1], k, v, torch.zeros((1, 1), dtype=torch.int32), [k.shape[1]], 1)
            assert rel_l2(out[b], ref[0]) <= OUT_TOL
        cached = outs["kv_lens"].clone()
        free = free[int(outs["pages_used"]):].contiguous()
    assert kda.read_device_status(ws) == 0
