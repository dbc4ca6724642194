"""Plain forms of the calls around the paged cache (torch in 64 bits, Python loops), and inputs for them."""
import random

import torch

D = 128


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- rotary positions
def rotary_reference(x, positions, inv_freq, axes, interleaved, mscale=1.0):
    """(x turned [rows, H, D], and the size of what met in each channel) in fp64; positions [axes, rows]."""
    x, positions, w = x.detach().double().cpu(), positions.cpu().long(), inv_freq.detach().double().cpu()
    half = w.numel()
    # an exact product in two parts (19 + 12 bits of the position times 24 of the frequency), joined by the angles' sum
    high, low = positions >> 12 << 12, positions & 4095
    y, size = x.clone(), x.abs()
    for f in range(half):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        one = torch.ones(x.shape[0], dtype=torch.float64)
        p0, p1 = high[axes[f]].double() * w[f], low[axes[f]].double() * w[f]
        z = (torch.polar(one, p0) * torch.polar(one, p1) * mscale)[:, None]
        t = torch.complex(x[..., a], x[..., b]) * z
        y[..., a], y[..., b] = t.real, t.imag
        size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(mscale)
    return y, size


# ---------------------------------------------------------------- pages
def held(lens, table, page):
    """The places of the table that are in use: (row, column)."""
    return [(b, c) for b, n in enumerate(lens) for c in range(-(-max(n, 0) // page))]


def fork_reference(table, lens, parents, children, free, page):
    """(table, lens, src, dst, used, refused)"""
    table, lens = [list(r) for r in table], list(lens)
    src, dst, need, refused = [], [], 0, 0
    for p, c in zip(parents, children):
        src.append(-1)
        dst.append(-1)
        if p < 0 or c < 0:
            continue
        n = lens[p]
        if n % page:
            need += 1
            if need > len(free):
                refused += 1
                continue
            src[-1], dst[-1] = table[p][n // page], free[need - 1]
        table[c][:n // page] = table[p][:n // page]
        if n % page:
            table[c][n // page] = dst[-1]
        lens[c] = n
    return table, lens, src, dst, min(need, len(free)), refused


def free_reference(table, lens, page, num_pages):
    used = {table[b][c] for b, c in held(lens, table, page)}
    free = [i for i in range(num_pages) if i not in used]
    return free + [-1] * (num_pages - len(free)), len(free)


def compact_reference(table, lens, page, num_pages, room, old_new):
    """(new table, src, dst, free, number free); places that are not in use come from old_new."""
    used = sorted({table[b][c] for b, c in held(lens, table, page) if 0 <= table[b][c] < num_pages})
    n = len(used)
    moves = [i for i in used if i >= n]
    there = set(used)
    holes = [i for i in range(n) if i not in there]
    to = dict(zip(moves, holes))
    new = [list(r) for r in old_new]
    for b, c in held(lens, table, page):
        new[b][c] = to.get(table[b][c], table[b][c])
    pad = [-1] * (room - len(moves))
    return new, moves + pad, holes + pad, list(range(n, num_pages)) + [-1] * n, num_pages - n


def page_case(B, longest, page, seed, extra=1.3, shared=1, width=None):
    """(table, lens, number of pages): rows of random lengths over a random order of the pages; rows of one group of `shared`
    begin with the same pages."""
    r = random.Random(seed)
    lens = [r.choice([0, r.randint(0, longest), r.randint(0, longest)]) for _ in range(B)]
    counts = [-(-n // page) for n in lens]
    total = int(sum(counts) * extra) + 2
    ids = list(range(total))
    r.shuffle(ids)
    width = width or max(counts + [1]) + r.randrange(3)
    table, at = [], 0
    for b, n in enumerate(counts):
        row = ids[at:at + n]
        at += n
        if shared > 1 and b % shared:
            m = min(n, counts[b - b % shared]) // 2
            row[:m] = table[b - b % shared][:m]
        table.append(row + [r.choice([-7, 0, total + 5]) for _ in range(width - n)])
    return table, lens, total
