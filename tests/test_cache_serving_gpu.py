"""The calls around the paged cache as a serving loop makes them: prompts, samples forked from them with their recurrent states,
steps with rotary stores and attention over the shared prompts, requests that end, the cache compacted in between."""
import math

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, i32, rotary_reference
from hybrid_refs import rel_l2

pytestmark = pytest.mark.gpu

# As in the attention's tests: weights and output are rounded to bf16 once each.
OUT_TOL = 2 * 2.0 ** -8


class Serving:
    """Two attention layers and one layer of recurrent states, of at most `slots` requests."""

    def __init__(self, slots, pages, page, width, hq, hk, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.page, self.hq, self.hk, self.slots = page, hq, hk, slots
        self.cache = [[torch.zeros((pages, page, hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
        self.states = torch.zeros((slots, 2, D, D), device="cuda")
        self.table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.free = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.count = i32([0])
        self.freq = (10000.0 ** (-torch.arange(64) / 64)).float().cuda()
        self.ws = kda.make_workspace(nbytes=kda.shared_prefix_workspace_size(slots, 1, hq, hk, 3))
        self.history = [[[[], []] for _ in range(2)] for _ in range(slots)]   # a request's keys (turned) and values, by layer
        self.release([])

    def release(self, rows):
        kda.release_requests(self.table, self.lens, i32(rows), self.page, free_pages=self.free, num_free=self.count, workspace=self.ws)
        for r in rows:
            self.history[r] = [[[], []] for _ in range(2)]

    def fork(self, pairs):
        parents, children = i32([p for p, _ in pairs]), i32([c for _, c in pairs])
        src, dst, used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (len(pairs), len(pairs), 1))
        kda.fork_requests(self.table, self.lens, parents, children, self.free[:int(self.count)], self.page, copy_src=src,
                          copy_dst=dst, pages_used=used, workspace=self.ws)
        kda.copy_pages([x for layer in self.cache for x in layer], src, dst, workspace=self.ws)
        kda.copy_pages([self.states], parents, children, workspace=self.ws)   # a slot is a page
        for p, c in pairs:
            self.history[c] = [[list(x) for x in layer] for layer in self.history[p]]
        self.release([])

    def compact(self):
        n = self.free.numel()
        src, dst = (torch.zeros(n // 2, dtype=torch.int32, device="cuda") for _ in range(2))
        kda.compact_pages(self.table, self.lens, self.page, new_table=self.table, copy_src=src, copy_dst=dst, free_pages=self.free,
                          num_free=self.count, workspace=self.ws)
        kda.copy_pages([x for layer in self.cache for x in layer], src, dst, workspace=self.ws)
        return n - int(self.count)

    def step(self, new, groups=None):
        """new: tokens of every request; groups: (first request, requests, shared tokens) for the attention, or none."""
        rows = sum(new) + 5
        outs = {"cu_seqlens": torch.zeros(self.slots + 1, dtype=torch.int32, device="cuda"),
                "kv_lens": torch.zeros(self.slots, dtype=torch.int32, device="cuda"),
                "positions": torch.zeros(rows, dtype=torch.int32, device="cuda"),
                "slot_map": torch.zeros(rows, dtype=torch.int64, device="cuda"), "pages_used": i32([0])}
        kda.step_tables(self.table, self.lens, i32(new), self.free[:int(self.count)], self.page, workspace=self.ws, **outs)
        cu = outs["cu_seqlens"].tolist()
        got = []
        for layer, (kp, vp) in enumerate(self.cache):
            q, k, v = (torch.randn((rows, h, D), generator=self.g, device="cuda").bfloat16() for h in (self.hq, self.hk, self.hk))
            turned = kda.rotary_to_pages(q, k, v, outs["positions"], outs["slot_map"], self.freq, kp, vp, workspace=self.ws)
            want, size = rotary_reference(q[:cu[-1]], outs["positions"][None, :cu[-1]], self.freq, [0] * 64, False)
            bound = 2.0 ** -8 * (want.abs() + 2.0 ** -21 * size) + 2.0 ** -21 * size + 1e-38
            assert ((turned[:cu[-1]].double().cpu() - want).abs() <= bound).all()
            key, _ = rotary_reference(k[:cu[-1]], outs["positions"][None, :cu[-1]], self.freq, [0] * 64, False)
            for b in range(self.slots):
                for t in range(cu[b], cu[b + 1]):
                    self.history[b][layer][0].append(key[t].bfloat16())
                    self.history[b][layer][1].append(v[t].cpu())
            if groups is not None and all(n <= 1 for n in new):
                last = torch.zeros((self.slots, self.hq, D), dtype=torch.bfloat16, device="cuda")
                for b in range(self.slots):
                    if new[b]:
                        last[b] = turned[cu[b]]
                lens = torch.where(i32(new) > 0, outs["kv_lens"], 0)
                starts, shared = [0], []
                for first, count, n in groups:
                    assert first == starts[-1]
                    starts.append(first + count)
                    shared.append(n)
                got.append((last, lens, kda.shared_prefix_attention(last, kp, vp, self.table, lens, i32(shared), i32(starts),
                                                                    workspace=self.ws)[0]))
        self.lens.copy_(outs["kv_lens"])
        for layer, (q, lens, out) in enumerate(got):
            for b, n in enumerate(lens.tolist()):
                if n == 0:
                    assert (out[b] == 0).all()
                    continue
                k, v = (torch.stack(x).double() for x in self.history[b][layer])
                assert k.shape[0] == n
                group = self.hq // self.hk
                for h in range(self.hk):
                    z = q[b, h * group:(h + 1) * group].double().cpu() @ k[:, h].T / math.sqrt(D)
                    ref = torch.softmax(z, -1) @ v[:, h]
                    # (a key may be off by a rounding the other way: half a step of bf16 more)
                    assert rel_l2(out[b, h * group:(h + 1) * group], ref) <= 2 * OUT_TOL
        self.release([])
        assert kda.read_device_status(self.ws) == 0


@pytest.mark.parametrize("width", [64, 30000])
def test_serving_loop(width):
    """With a narrow table every request attends alone; with a wide one the prompts are shared."""
    s = Serving(slots=12, pages=120, page=16, width=width, hq=8, hk=2, seed=1)
    # two prompts, in requests 0 and 6
    new = [0] * 12
    new[0], new[6] = 333, 97
    s.step(new)
    s.states[0].normal_(generator=s.g)
    s.states[6].normal_(generator=s.g)
    s.fork([(0, c) for c in range(1, 6)] + [(6, c) for c in range(7, 11)])
    for c in range(1, 6):
        assert torch.equal(s.states[c], s.states[0])
    used = len(set(x for b in range(12) for x in s.table[b, :-(-int(s.lens[b]) // 16)].tolist()))
    # 333 tokens: 20 pages in common and one for each of six; 97: 6 and 5
    assert used == 20 + 6 + 6 + 5 and int(s.count) == 120 - used
    groups = [(0, 6, 333), (6, 5, 97), (11, 1, 0)]
    for _ in range(3):
        s.step([1] * 11 + [0], groups)
    s.release([0, 2, 8])
    assert s.compact() == int(len(set(x for b in range(12) for x in s.table[b, :-(-int(s.lens[b]) // 16)].tolist())))
    live = [0, 1, 0, 1, 1, 1, 1, 1, 0, 1, 1, 0]
    for _ in range(2):
        s.step(live, groups)
    # a freed slot takes a sample of a sample, another a new prompt
    s.fork([(3, 2)])
    live[2] = 1
    s.step([n if b != 11 else 40 for b, n in enumerate(live)])
    s.step([n if b != 11 else 1 for b, n in enumerate(live)], groups)
    s.release(list(range(12)))
    assert int(s.count) == 120 and s.compact() == 0
