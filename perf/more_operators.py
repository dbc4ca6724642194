"""Measured operators around the paged cache: rotary positions of one or several axes with the step's keys and values
stored into their pages, attention for batches whose requests share long prefixes, and the pages' own operations (forking
requests, releasing them, compacting the cache, copying pages of every layer).

Every operator has its plain form here: elementary torch operations in fp32 (fp64 for the angles of far positions), rounded
once at the end.  With ``own`` set, ``run`` makes the calls a user makes of this package instead.

Notation.  Request b has seq_lens[b] tokens in the cache, its last T new; token j of it lies in page
block_table[b, j // page] at row j % page.
    rotary:    theta = positions[axis of frequency f, i] inv_freq[f];  (a, b) -> m (a cos - b sin, b cos + a sin)
    attention: out = softmax(q k^T / sqrt(128)) v over the tokens a new token sees, lse = log of the weights' sum
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch: one token per request, far positions, three padding rows of a captured bucket
        {"name": "rotary_61of64_h16_k2", "op": "rotary", "tokens": 61, "padding": 3, "axes": 1, "hq": 16, "hk": 2,
         "rot": 128, "page": 16, "interleaved": False, "fused": False, "far": 1000000},
        # a prompt of video frames: time, height and width, one fused projection of q, k and v
        {"name": "rotary_video_9001_h32_k8", "op": "rotary", "tokens": 9001, "padding": 0, "axes": 3, "hq": 32, "hk": 8,
         "rot": 128, "page": 64, "interleaved": False, "fused": True, "far": 200000},
        # one prompt, four samples of it, two layers: latency
        {"name": "fork_1to4_2layers", "op": "fork", "prompts": 1, "copies": 4, "longest": 333, "layers": 2, "hk": 2,
         "page": 16, "lens_seed": 1},
        # 48 prompts, five samples of each: table rows shared, the last pages of every layer copied
        {"name": "fork_48to240_8layers", "op": "fork", "prompts": 48, "copies": 5, "longest": 2500, "layers": 8, "hk": 4,
         "page": 64, "lens_seed": 2},
        # a few requests of a decode batch end
        {"name": "release_5of64", "op": "release", "reqs": 64, "done": 5, "longest": 8192, "group": 1, "page": 16,
         "lens_seed": 3},
        # a fifth of a large batch ends, groups of eight share their prompts' pages
        {"name": "release_100of512", "op": "release", "reqs": 512, "done": 100, "longest": 30000, "group": 8, "page": 16,
         "lens_seed": 4},
        # a small fragmented cache
        {"name": "compact_12_2layers", "op": "compact", "reqs": 12, "longest": 900, "layers": 2, "hk": 2, "page": 16,
         "fill": 70, "lens_seed": 5},
        # a cache filled to 60 percent, six layers, so that its upper part can be given away
        {"name": "compact_60_6layers", "op": "compact", "reqs": 60, "longest": 3100, "layers": 6, "hk": 4, "page": 32,
         "fill": 60, "lens_seed": 6},
        # four samples of one short prompt early in their generation: latency
        {"name": "prefix_4x500_h16_k2", "op": "prefix", "groups": 1, "fewest": 4, "most": 4, "steps": 1, "shared": 500,
         "least_shared": 500, "longest": 40, "hq": 16, "hk": 2, "page": 16, "lens_seed": 7},
        # 64 samples of one prompt, each some hundred tokens further
        {"name": "prefix_64x8192_h16_k2", "op": "prefix", "groups": 1, "fewest": 64, "most": 64, "steps": 1,
         "shared": 8192, "least_shared": 8192, "longest": 700, "hq": 16, "hk": 2, "page": 64, "lens_seed": 8},
        # a mixed batch: seven prompts of very different lengths, 1 to 24 requests on each, drafts of four tokens
        {"name": "prefix_7groups_x4_h16_k2", "op": "prefix", "groups": 7, "fewest": 1, "most": 24, "steps": 4,
         "shared": 20000, "least_shared": 100, "longest": 300, "hq": 16, "hk": 2, "page": 48, "lens_seed": 9},
        # many requests on one very long document: work is bound by the products
        {"name": "prefix_192x40000_h32_k4", "op": "prefix", "groups": 1, "fewest": 192, "most": 192, "steps": 1,
         "shared": 40000, "least_shared": 40000, "longest": 400, "hq": 32, "hk": 4, "page": 64, "lens_seed": 10},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "fork", "release", "compact", "prefix", "prefix"])
    seed = rng.randrange(1 << 20)
    if op == "rotary":
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5, 8])
        return {"op": op, "tokens": _log_int(rng, 1, 9001 * 40 // (hq + 2 * hk + 10)), "padding": rng.choice([0, 0, 5]),
                "axes": rng.choice([1, 1, 2, 3, 4]), "hq": hq, "hk": hk, "rot": rng.choice([128, 128, 96, 64, 32]),
                "page": rng.choice([1, 16, 24, 64, 256]), "interleaved": rng.random() < 0.4, "fused": rng.random() < 0.5,
                "far": _log_int(rng, 10, 1000000)}
    if op == "fork":
        hk, page = rng.choice([1, 2, 4]), rng.choice([1, 16, 24, 64])
        prompts, copies, layers = _log_int(rng, 1, 48), rng.randrange(1, 9), rng.randrange(1, 9)
        longest = min(_log_int(rng, 1, 2500), 2500 * 48 * 8 * 4 // (prompts * layers * hk))
        copies = max(1, min(copies, 240 * 8 * 4 * 64 // (prompts * layers * hk * page)))
        return {"op": op, "prompts": prompts, "copies": copies, "longest": longest, "layers": layers, "hk": hk, "page": page,
                "lens_seed": seed}
    if op == "release":
        reqs = _log_int(rng, 1, 512)
        return {"op": op, "reqs": reqs, "done": rng.randrange(0, reqs + 1), "longest": _log_int(rng, 1, 30000),
                "group": rng.choice([1, 1, 4, 8]), "page": rng.choice([16, 48, 64, 256]), "lens_seed": seed}
    if op == "compact":
        hk, page, layers = rng.choice([1, 2, 4]), rng.choice([4, 16, 32, 64]), rng.randrange(1, 7)
        reqs = _log_int(rng, 1, 60)
        longest = min(_log_int(rng, 1, 3100), 60 * 3100 * 4 * 6 // (reqs * hk * layers))
        return {"op": op, "reqs": reqs, "longest": longest, "layers": layers, "hk": hk, "page": page,
                "fill": rng.randrange(30, 100), "lens_seed": seed}
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 4, 5, 8])
    groups, most, steps = rng.choice([1, 1, 2, 3, 7]), _log_int(rng, 2, 192), rng.choice([1, 1, 1, 2, 4])
    most = max(2, min(most, 192 * 32 // (groups * hq * steps)))
    shared = min(_log_int(rng, 16, 40000), 192 * 32 * 40000 // (groups * most * steps * hq))
    return {"op": op, "groups": groups, "fewest": rng.choice([1, most]), "most": most, "steps": steps, "shared": shared,
            "least_shared": rng.choice([max(1, shared // 8), shared]), "longest": _log_int(rng, 4, 400),
            "hq": hq, "hk": hk, "page": rng.choice([1, 16, 24, 64, 256]), "lens_seed": seed}


def _pages(tokens, page):
    return -(-tokens // page)


def _lens(case, count, shortest, longest):
    """Lengths of a case, the longest among them."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(shortest, longest) for _ in range(count)]
    lens[r.randrange(count)] = longest
    return lens


def _batch(case):
    """(shared tokens of each group, its requests, own tokens of every request) of a case of shared prefixes."""
    r = random.Random(case["lens_seed"])
    shared = [r.randint(case["least_shared"], case["shared"]) for _ in range(case["groups"])]
    sizes = [r.randint(case["fewest"], case["most"]) for _ in range(case["groups"])]
    shared[0], sizes[0] = case["shared"], case["most"]
    tails = [max(case["steps"], r.randint(1, case["longest"])) for _ in range(sum(sizes))]
    return shared, sizes, tails


def _shared_pages(case):
    """(pages of every request's row, pages that a group of rows has in common) of a release case."""
    lens = _lens(case, case["reqs"], 1, case["longest"])
    count = [_pages(n, case["page"]) for n in lens]
    common = [min(count[g:g + case["group"]]) * 3 // 4 if case["group"] > 1 else 0
              for g in range(0, case["reqs"], case["group"])]
    return lens, count, common


def _live_pages(case):
    return sum(_pages(n, case["page"]) for n in _lens(case, case["reqs"], 1, case["longest"]))


def work(case):
    op, page = case["op"], case.get("page")
    if op == "rotary":
        t, hq, hk = case["tokens"], case["hq"], case["hk"]
        return {"bytes": t * (4 * hq * D + 8 * hk * D + 4 * case["axes"] + 8) + 8 * case["padding"] + 2 * case["rot"],
                "flops": t * (hq + hk) * 3 * case["rot"]}
    if op == "fork":
        lens = _lens(case, case["prompts"], 1, case["longest"])
        rows = sum(4 * _pages(n, page) * (1 + case["copies"]) for n in lens)
        parts = sum(n % page > 0 for n in lens) * case["copies"]
        return {"bytes": rows + parts * case["layers"] * 2 * page * case["hk"] * D * 4 + 28 * case["prompts"] * case["copies"],
                "flops": 0}
    if op == "release":
        _, count, common = _shared_pages(case)
        total = sum(count)
        pages = total - sum(c * (len(count[g * case["group"]:(g + 1) * case["group"]]) - 1) for g, c in enumerate(common))
        kept = total * (case["reqs"] - case["done"]) // case["reqs"]
        return {"bytes": 4 * kept + 4 * (pages * 5 // 4) + 8 * case["reqs"], "flops": 0}
    if op == "compact":
        live = _live_pages(case)
        size = live * 100 // case["fill"] + 1
        moved = live * (size - live) // size
        return {"bytes": 8 * live + 4 * size + moved * (8 + case["layers"] * 2 * page * case["hk"] * D * 4) + 4 * case["reqs"],
                "flops": 0}
    shared, sizes, tails = _batch(case)
    t, hq, hk = case["steps"], case["hq"], case["hk"]
    b = sum(sizes)
    tokens = sum(shared) + sum(tails)
    pairs = t * sum(p * n for p, n in zip(shared, sizes)) + sum(t * n - t * (t - 1) // 2 for n in tails)
    return {"bytes": tokens * hk * D * 4 + b * t * hq * (D * 4 + 4) + 4 * _pages(tokens, page) + 4 * b,
            "flops": pairs * hq * 4 * D}


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(gen, pages, page, hk):
    return torch.randn((pages, page, hk, D), generator=gen, device="cuda", dtype=torch.bfloat16)


def _rows_of(order, counts, width):
    """A block table: row r holds the next counts[r] ids of `order`, the rest is 0."""
    n = torch.tensor(counts, device="cuda")
    first = torch.cumsum(n, 0) - n
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=order.shape[0] - 1)
    return torch.where(col < n[:, None], order[at], torch.zeros_like(order[at])).contiguous()


def _prepare_rotary(case, gen, s):
    rows, hq, hk, page, axes, half = (case["tokens"] + case["padding"], case["hq"], case["hk"], case["page"], case["axes"],
                                      case["rot"] // 2)
    qkv = torch.randn((rows, hq + 2 * hk, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    parts = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    s["q"], s["k"], s["v"] = parts if case["fused"] else (x.contiguous() for x in parts)
    # a frame of tokens has one time, its rows heights, their columns widths; with one axis every token a place of its own
    i = torch.arange(rows, device="cuda")
    if axes > 1:
        side = max(1, int(math.sqrt(rows) / 2))
        place = [i // (side * side), i // side % side, i % side, i % 7]
    else:
        place = [torch.randint(0, case["far"], (rows,), generator=gen, device="cuda")]
    start = torch.randint(0, max(1, case["far"] - rows), (1,), generator=gen, device="cuda")
    s["positions"] = torch.stack([p + (start if axes > 1 else 0) for p in place[:axes]]).to(torch.int32)
    live = torch.arange(rows, device="cuda") < case["tokens"]
    s["positions"][:, ~live] = 0
    s["inv_freq"] = 1000000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
    s["axes"] = bytes(f * axes // half for f in range(half))     # equal sections, the fastest frequencies the first axis's
    pages = _pages(rows, page) * 2 + 1
    s["slots"] = torch.where(live, torch.randperm(pages * page, generator=gen, device="cuda")[:rows], -1)
    s["k_pages"], s["v_pages"] = _cache(gen, pages, page, hk), _cache(gen, pages, page, hk)
    s["out"] = torch.zeros((rows, hq, D), dtype=torch.bfloat16, device="cuda")


def _prepare_fork(case, gen, s):
    page, prompts, copies = case["page"], case["prompts"], case["copies"]
    lens = _lens(case, prompts, 1, case["longest"])
    count = [_pages(n, page) for n in lens]
    total = sum(count)
    order = torch.randperm(total + prompts * copies + 3, generator=gen, device="cuda").to(torch.int32)
    s["table"] = torch.zeros((prompts * (1 + copies), max(count) + 2), dtype=torch.int32, device="cuda")
    s["table"][:prompts] = _rows_of(order[:total], count, max(count) + 2)
    s["lens"] = _i32(lens + [0] * (prompts * copies))
    s["parents"] = _i32([p for p in range(prompts) for _ in range(copies)])
    s["children"] = _i32(list(range(prompts, prompts * (1 + copies))))
    s["free"] = order[total:].contiguous()
    for name in ("src", "dst"):
        s[name] = torch.zeros(prompts * copies, dtype=torch.int32, device="cuda")
    s["used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["buffers"] = [_cache(gen, order.shape[0], page, case["hk"]) for _ in range(2 * case["layers"])]


def _prepare_release(case, gen, s):
    lens, count, common = _shared_pages(case)
    width, group = max(count) + 3, case["group"]
    total = sum(count)
    order = torch.randperm(total + total // 4 + 1, generator=gen, device="cuda").to(torch.int32)
    table = _rows_of(order, count, width)
    # the rows of a group begin with its first row's pages
    first = torch.arange(case["reqs"], device="cuda") // group * group
    shared = torch.tensor([common[b // group] for b in range(case["reqs"])], device="cuda")
    s["table"] = torch.where(torch.arange(width, device="cuda") < shared[:, None], table[first], table).contiguous()
    s["lens"] = _i32(lens)
    s["rows"] = torch.randperm(case["reqs"], generator=gen, device="cuda")[:case["done"]].to(torch.int32)
    s["free"] = torch.zeros(order.shape[0], dtype=torch.int32, device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _prepare_compact(case, gen, s):
    lens = _lens(case, case["reqs"], 1, case["longest"])
    count = [_pages(n, case["page"]) for n in lens]
    live = sum(count)
    size = live * 100 // case["fill"] + 1
    order = torch.randperm(size, generator=gen, device="cuda").to(torch.int32)
    s["table"] = _rows_of(order[:live], count, max(count) + 1)
    s["lens"] = _i32(lens)
    s["new_table"] = torch.zeros_like(s["table"])
    for name, n in (("src", size // 2), ("dst", size // 2), ("free", size), ("count", 1)):
        s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["buffers"] = [_cache(gen, size, case["page"], case["hk"]) for _ in range(2 * case["layers"])]


def _prepare_prefix(case, gen, s):
    shared, sizes, tails = _batch(case)
    t, hq, hk, page = case["steps"], case["hq"], case["hk"], case["page"]
    group = [g for g, n in enumerate(sizes) for _ in range(n)]
    lens = [shared[g] + n for g, n in zip(group, tails)]
    # whole pages of a prompt are one request's and the others' too; the rest of every request lies in pages of its own
    whole = [p // page for p in shared]
    own_pages = [_pages(n, page) - whole[g] for g, n in zip(group, lens)]
    width = max(_pages(n, page) for n in lens)
    total = sum(whole) + sum(own_pages)
    order = torch.randperm(total + 2, generator=gen, device="cuda").to(torch.int32)[:total]
    prompt = _rows_of(order[:max(1, sum(whole))], whole, max(max(whole), 1))
    tail = _rows_of(order[sum(whole):], own_pages, max(own_pages))
    at, g = torch.arange(width, device="cuda"), torch.tensor(group, device="cuda")
    w = torch.tensor(whole, device="cuda")[g][:, None]
    head = prompt[g].gather(1, at.clamp(max=prompt.shape[1] - 1).expand(len(group), width))
    rest = tail.gather(1, (at - w).clamp(0, tail.shape[1] - 1))
    s["table"] = torch.where(at < w, head, rest).contiguous()
    s["k_pages"], s["v_pages"] = _cache(gen, total + 2, page, hk), _cache(gen, total + 2, page, hk)
    # what is left of a prompt behind its whole pages: copies of it in every request
    start = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    first = torch.tensor(start[:-1], device="cuda")[g]
    left = (torch.tensor(shared, device="cuda")[g] % page)[:, None, None, None]
    mine = s["table"].gather(1, w)[:, 0].long()
    place = torch.arange(page, device="cuda")[:, None, None]
    for x in (s["k_pages"], s["v_pages"]):
        x[mine] = torch.where(place < left, x[mine[first]], x[mine])
    s["q"] = 1.5 * torch.randn((len(group) * t, hq, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["lens"], s["shared"], s["starts"] = _i32(lens), _i32(shared), _i32(start)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((len(group) * t, hq), dtype=torch.float32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"rotary": _prepare_rotary, "fork": _prepare_fork, "release": _prepare_release, "compact": _prepare_compact,
     "prefix": _prepare_prefix}[case["op"]](case, gen, s)
    if own:   # the workspace that a serving program keeps
        import kda_linear_attention_bounded_gb300 as kda
        s["ws"] = kda.make_workspace()
        if case["op"] == "prefix":
            s["ws"] = kda.make_workspace(nbytes=kda.shared_prefix_workspace_size(
                s["lens"].shape[0], case["steps"], case["hq"], case["hk"], case["groups"]))
    return s


# ---------------------------------------------------------------- plain forms
def _turned(x, cos, sin, rot, interleaved):
    x = x.float()
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    y = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotary(s):
    rot, page = s["case"]["rot"], s["case"]["page"]
    axis = torch.tensor(list(s["axes"]), device=s["q"].device)
    theta = s["positions"].double()[axis] * s["inv_freq"].double()[:, None]            # [frequencies, rows]
    cos, sin = torch.cos(theta).float().T[:, None], torch.sin(theta).float().T[:, None]
    live = s["slots"] >= 0
    q = _turned(s["q"], cos, sin, rot, s["case"]["interleaved"]).to(torch.bfloat16)
    s["out"].copy_(torch.where(live[:, None, None], q, s["out"]))
    k = _turned(s["k"], cos, sin, rot, s["case"]["interleaved"]).to(torch.bfloat16)
    at = s["slots"][live]
    s["k_pages"][at // page, at % page] = k[live]
    s["v_pages"][at // page, at % page] = s["v"][live]
    return s["out"], s["k_pages"], s["v_pages"]


def _plain_copies(buffers, src, dst):
    live = (src >= 0) & (dst >= 0)
    a, b = src[live].long(), dst[live].long()
    return [x.index_copy_(0, b, x[a]) for x in buffers]


def _plain_fork(s):
    page, table = s["case"]["page"], s["table"]
    p, c = s["parents"].long(), s["children"].long()
    n = s["lens"][p]
    whole, part = n // page, n % page > 0
    taken = torch.cumsum(part, 0) - 1
    fresh = s["free"][taken.clamp(min=0)]
    col = torch.arange(table.shape[1], device=table.device)
    from_parent = torch.where(col < whole[:, None], table[p], table[c])
    table[c] = torch.where((col == whole[:, None]) & part[:, None], fresh[:, None], from_parent)
    last = table[p].gather(1, whole.long()[:, None].clamp(max=table.shape[1] - 1))[:, 0]
    s["src"].copy_(torch.where(part, last, -1))
    s["dst"].copy_(torch.where(part, fresh, -1))
    s["lens"][c] = n
    s["used"].copy_(part.sum())
    return table, s["lens"], s["src"], s["dst"], s["used"], _plain_copies(s["buffers"], s["src"], s["dst"])


def _marks(table, lens, page, count):
    """Which of the pages the requests hold, and which places of the table are theirs."""
    held = torch.arange(table.shape[1], device=table.device) < ((lens + page - 1) // page)[:, None]
    used = torch.zeros(count + 1, dtype=torch.bool, device=table.device)
    used[torch.where(held, table, count).long().flatten()] = True
    return used[:count], held


def _plain_release(s):
    s["lens"][s["rows"].long()] = 0
    size = s["free"].shape[0]
    used, _ = _marks(s["table"], s["lens"], s["case"]["page"], size)
    ids = torch.arange(size, device=used.device)
    rank = torch.cumsum(~used, 0) - 1
    free = torch.full((size + 1,), -1, dtype=torch.int32, device=used.device)
    free[torch.where(used, size, rank)] = torch.where(used, -1, ids).to(torch.int32)
    s["free"].copy_(free[:size])
    s["count"].copy_((~used).sum())
    return s["lens"], s["free"], s["count"]


def _plain_compact(s):
    size, room = s["free"].shape[0], s["src"].shape[0]
    used, held = _marks(s["table"], s["lens"], s["case"]["page"], size)
    ids = torch.arange(size, device=used.device)
    live = used.sum()
    move, hole = used & (ids >= live), ~used & (ids < live)
    move_rank, hole_rank = torch.cumsum(move, 0) - 1, torch.cumsum(hole, 0) - 1
    lists = torch.full((2, room + 1), -1, dtype=torch.int32, device=used.device)
    lists[0, torch.where(move, move_rank, room)] = torch.where(move, ids, -1).to(torch.int32)
    lists[1, torch.where(hole, hole_rank, room)] = torch.where(hole, ids, -1).to(torch.int32)
    s["src"].copy_(lists[0, :room])
    s["dst"].copy_(lists[1, :room])
    new_id = torch.where(move, lists[1][move_rank.clamp(min=0)].long(), ids)
    table = new_id[torch.where(held, s["table"], 0).long()].to(torch.int32)
    s["new_table"].copy_(torch.where(held, table, s["new_table"]))
    s["count"].copy_(size - live)
    s["free"].copy_(torch.where(ids < size - live, ids + live, -1))
    return s["new_table"], s["src"], s["dst"], s["free"], s["count"], _plain_copies(s["buffers"], s["src"], s["dst"])


def _plain_prefix(s):
    """The groups' prefixes gathered once each and met by all the group's queries, the requests' own tokens gathered for
    each, one softmax over both."""
    t, hq, hk, page = (s["case"][n] for n in ("steps", "hq", "hk", "page"))
    dev, group = s["q"].device, hq // hk
    table, starts, shared, lens = s["table"].long(), s["starts"].long(), s["shared"].long(), s["lens"].long()
    b, groups = lens.shape[0], shared.shape[0]
    mine = torch.bucketize(torch.arange(b, device=dev), starts, right=True) - 1      # a request's group
    q = s["q"].float().view(b, t, hk, group, D).permute(0, 2, 1, 3, 4).reshape(b, hk, t * group, D)

    def tokens(pages, rows, pos):   # keys or values of the tokens pos of table rows `rows`
        at = table[rows[:, None], (pos // page).clamp(max=table.shape[1] - 1)]
        return pages[at, pos % page].float()                                         # [rows, n, hk, D]

    # the prefixes: [groups, hk, members x rows, longest prefix]
    members, longest = (starts[1:] - starts[:-1]).amax(), shared.amax()
    slot = torch.arange(b, device=dev) - starts[mine]
    grouped = torch.zeros((groups, int(members), hk, t * group, D), device=dev)
    grouped[mine, slot] = q
    grouped = grouped.transpose(1, 2).reshape(groups, hk, -1, D)
    pos = torch.arange(int(longest), device=dev).expand(groups, -1)
    k = tokens(s["k_pages"], starts[:-1], pos).permute(0, 2, 3, 1)
    score = (grouped @ k) * SCALE
    del k
    score = score.masked_fill((pos >= shared[:, None])[:, None, None], -math.inf)
    # the requests' own tokens: [b, hk, rows, longest rest]
    rest = (lens - shared[mine]).amax()
    pos2 = shared[mine][:, None] + torch.arange(int(rest), device=dev)
    last = lens[:, None] - t + torch.arange(t, device=dev)
    seen = (pos2[:, None] <= last[..., None])[:, None, :, None].expand(b, 1, t, group, int(rest)).reshape(b, 1, t * group, -1)
    score2 = (q @ tokens(s["k_pages"], torch.arange(b, device=dev), pos2).permute(0, 2, 3, 1)) * SCALE
    score2 = score2.masked_fill(~seen, -math.inf)

    def of_requests(x):   # [groups, hk, members rows, n] -> [b, hk, rows, n]
        return x.view(groups, hk, int(members), t * group, -1).transpose(1, 2)[mine, slot]

    def of_groups(x):     # and back
        y = torch.zeros((groups, int(members), *x.shape[1:]), device=dev)
        y[mine, slot] = x
        return y.transpose(1, 2).reshape(groups, hk, -1, x.shape[-1])

    top = torch.maximum(of_requests(score.amax(-1, keepdim=True)), score2.amax(-1, keepdim=True))
    p, p2 = torch.exp(score - of_groups(top)), torch.exp(score2 - top)
    del score, score2
    v = tokens(s["v_pages"], starts[:-1], pos).permute(0, 2, 1, 3)
    v2 = tokens(s["v_pages"], torch.arange(b, device=dev), pos2).permute(0, 2, 1, 3)
    total = of_requests(p.sum(-1, keepdim=True)) + p2.sum(-1, keepdim=True)
    o = (of_requests(p @ v) + p2 @ v2) / total

    def rows(x):   # [b, hk, t group, n] -> [b t, hq, n]
        return x.view(b, hk, t, group, -1).permute(0, 2, 1, 3, 4).reshape(b * t, hq, -1)

    s["out"].copy_(rows(o))
    s["lse"].copy_(rows(top + torch.log(total))[..., 0])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- the framework's calls
def _own_run(s):
    import kda_linear_attention_bounded_gb300 as kda

    op, page = s["op"], s["case"]["page"]
    if op == "rotary":
        out = kda.rotary_to_pages(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_pages"],
                                  s["v_pages"], axes=s["axes"], interleaved=s["case"]["interleaved"], out=s["out"],
                                  workspace=s["ws"])
        return out, s["k_pages"], s["v_pages"]
    if op == "fork":
        kda.fork_requests(s["table"], s["lens"], s["parents"], s["children"], s["free"], page, copy_src=s["src"],
                          copy_dst=s["dst"], pages_used=s["used"], workspace=s["ws"])
        kda.copy_pages(s["buffers"], s["src"], s["dst"], workspace=s["ws"])
        return s["table"], s["lens"], s["src"], s["dst"], s["used"], s["buffers"]
    if op == "release":
        kda.release_requests(s["table"], s["lens"], s["rows"], page, free_pages=s["free"], num_free=s["count"],
                             workspace=s["ws"])
        return s["lens"], s["free"], s["count"]
    if op == "compact":
        kda.compact_pages(s["table"], s["lens"], page, new_table=s["new_table"], copy_src=s["src"], copy_dst=s["dst"],
                          free_pages=s["free"], num_free=s["count"], workspace=s["ws"])
        kda.copy_pages(s["buffers"], s["src"], s["dst"], workspace=s["ws"])
        return s["new_table"], s["src"], s["dst"], s["free"], s["count"], s["buffers"]
    return kda.shared_prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["shared"], s["starts"],
                                       s["case"]["steps"], out=s["out"], lse=s["lse"], workspace=s["ws"])


def run(state):
    if own:
        return _own_run(state)
    return {"rotary": _plain_rotary, "fork": _plain_fork, "release": _plain_release, "compact": _plain_compact,
            "prefix": _plain_prefix}[state["op"]](state)


# ---------------------------------------------------------------- 64-bit definitions
def _exact_rotary(s, case):
    half, page = case["rot"] // 2, case["page"]
    out, pages = s["out"].double(), [s["k_pages"].double(), s["v_pages"].double()]
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    q, k = s["q"][live].double(), s["k"][live].double()
    for f in range(half):
        a, b = (2 * f, 2 * f + 1) if case["interleaved"] else (f, f + half)
        theta = s["positions"][s["axes"][f], live].double() * s["inv_freq"][f].double()
        z = torch.polar(torch.ones_like(theta), theta)[:, None]
        for x in (q, k):
            w = torch.complex(x[..., a], x[..., b]) * z
            x[..., a], x[..., b] = w.real, w.imag
    out[live] = q
    at = s["slots"][live]
    pages[0].flatten(0, 1)[at] = k
    pages[1].flatten(0, 1)[at] = s["v"][live].double()
    return out, pages[0], pages[1]


def exact(case, seed):
    if case["op"] not in ("rotary", "prefix"):
        return None
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    t, hq, hk, page = case["steps"], case["hq"], case["hk"], case["page"]
    group = hq // hk
    out = torch.empty((s["q"].shape[0], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["q"].shape[0], hq), dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        pos = torch.arange(n, device="cuda")
        at = s["table"][i].long()[pos // page]
        for h in range(hk):
            kh, vh = s["k_pages"][at, pos % page, h].double(), s["v_pages"][at, pos % page, h].double()
            for j in range(t):
                last = n - t + j + 1
                mine = slice(h * group, (h + 1) * group)
                z = s["q"][i * t + j, mine].double() @ kh[:last].T / math.sqrt(D)
                lse[i * t + j, mine] = torch.logsumexp(z, -1)
                out[i * t + j, mine] = torch.softmax(z, -1) @ vh[:last]
    return out, lse
