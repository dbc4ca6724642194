"""Measured operators of the hybrid-layer set: the gated delta rule (chunked prefill, recurrent decode and verify),
attention of new tokens over a paged key-value cache, and the step tables (page tables and slot maps) built on the GPU.

Every operator has its plain form here: elementary torch operations in fp32 (fp64 for the running sums of
log-decays, whose differences are exponentiated), rounded once at the end.  With ``own`` set, ``run`` makes the
calls a user makes of this package instead.

Notation of the gated delta rule, per value head h (its key head is h // (Hv / Hk)) and token t:
    q^, k^     = q, k / sqrt(sum of squares + 1e-6)
    beta       = sigmoid(beta_logit),  lambda = -exp(A_log) softplus(a + dt_bias)
    S_t        = (I - beta k^ k^T) e^lambda S_{t-1} + beta k^ v^T,   o_t = S_t^T q^ / sqrt(128)
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
CHUNK = 64
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt of one small layer: launch latency counts
        {"name": "gdn_prefill_1x256_h2", "op": "gdn_prefill", "seqs": 1, "longest": 256, "shortest": 256, "hk": 2,
         "hv": 2, "initial": False, "lens_seed": 0},
        # a full prefill batch that continues cached prefixes (initial states from the pool)
        {"name": "gdn_prefill_2048x8_h16", "op": "gdn_prefill", "seqs": 8, "longest": 2048, "shortest": 2048,
         "hk": 16, "hv": 16, "initial": True, "lens_seed": 0},
        # one long prompt, key heads shared by two value heads: a few long serial chains
        {"name": "gdn_prefill_16384x1_h16_k8", "op": "gdn_prefill", "seqs": 1, "longest": 16384, "shortest": 16384,
         "hk": 8, "hv": 16, "initial": False, "lens_seed": 0},
        # a ragged batch of prompts, odd lengths, key heads shared by four value heads
        {"name": "gdn_prefill_ragged_h32_k8", "op": "gdn_prefill", "seqs": 13, "longest": 2500, "shortest": 1,
         "hk": 8, "hv": 32, "initial": True, "lens_seed": 3},
        # plain decoding of one request
        {"name": "gdn_decode_1_h16", "op": "gdn_decode", "reqs": 1, "hk": 16, "hv": 16, "slots": 8},
        # plain decoding of a full batch, states updated in the pool
        {"name": "gdn_decode_64_h16", "op": "gdn_decode", "reqs": 64, "hk": 16, "hv": 16, "slots": 256},
        # speculative verify: three drafts plus the bonus token, every per-step state recorded
        {"name": "gdn_verify_64x4_h16_k8", "op": "gdn_verify", "reqs": 64, "steps": 4, "hk": 8, "hv": 16, "slots": 96},
        # one request early in its generation: latency
        {"name": "paged_1x257_h16_k2", "op": "paged", "reqs": 1, "steps": 1, "longest": 257, "shortest": 257,
         "hq": 16, "hk": 2, "page": 16, "lens_seed": 0},
        # a decode batch of very different context lengths
        {"name": "paged_64_to_8192_h16_k2", "op": "paged", "reqs": 64, "steps": 1, "longest": 8192, "shortest": 1,
         "hq": 16, "hk": 2, "page": 64, "lens_seed": 5},
        # speculative verify over long contexts, few requests: work is split over the cache's length
        {"name": "paged_5x4_to_131072_h16_k2", "op": "paged", "reqs": 5, "steps": 4, "longest": 131072,
         "shortest": 40000, "hq": 16, "hk": 2, "page": 16, "lens_seed": 7},
        # the tables of one decode step
        {"name": "tables_64x1", "op": "tables", "reqs": 64, "newest": 1, "fewest": 1, "cached": 8192, "page": 16,
         "lens_seed": 1},
        # the tables of a mixed step: decoding requests and prompt chunks of up to 2000 tokens
        {"name": "tables_512_mixed", "op": "tables", "reqs": 512, "newest": 2000, "fewest": 0, "cached": 30000,
         "page": 64, "lens_seed": 2},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdn_prefill", "gdn_prefill", "gdn_decode", "gdn_verify", "paged", "paged", "tables"])
    seed = rng.randrange(1 << 20)
    if op == "gdn_prefill":
        hv = rng.choice([2, 3, 8, 16, 32])
        hk = hv // rng.choice([g for g in (1, 2, 4) if hv % g == 0])
        seqs = _log_int(rng, 1, 24)
        longest = min(_log_int(rng, 1, 16384), max(64, 200000 // (seqs * hv)))
        return {"op": op, "seqs": seqs, "longest": longest, "shortest": rng.choice([1, longest]), "hk": hk, "hv": hv,
                "initial": rng.random() < 0.5, "lens_seed": seed}
    if op == "gdn_decode":
        hv = rng.choice([4, 7, 16, 32])
        reqs = min(_log_int(rng, 1, 256), 1024 // hv)
        return {"op": op, "reqs": reqs, "hk": hv // rng.choice([g for g in (1, 2, 4) if hv % g == 0]), "hv": hv,
                "slots": reqs + rng.randrange(1, 40)}
    if op == "gdn_verify":
        hv = rng.choice([4, 7, 16, 32])
        steps = rng.randrange(2, 9)
        reqs = min(_log_int(rng, 1, 128), max(1, 4096 // (hv * steps)))
        return {"op": op, "reqs": reqs, "steps": steps, "hk": hv // rng.choice([g for g in (1, 2, 4) if hv % g == 0]),
                "hv": hv, "slots": reqs + rng.randrange(1, 40)}
    if op == "paged":
        hk = rng.choice([1, 2, 4, 8])
        reqs = _log_int(rng, 1, 128)
        longest = min(_log_int(rng, 1, 131072), max(64, 900000 // (reqs * hk)))
        return {"op": op, "reqs": reqs, "steps": rng.choice([1, 1, 1, 2, 3, 4, 8]), "longest": max(longest, 8),
                "shortest": rng.choice([1, max(1, longest // 2)]), "hq": hk * rng.choice([1, 2, 4, 5, 8, 16]),
                "hk": hk, "page": rng.choice([1, 16, 24, 64, 256]), "lens_seed": seed}
    return {"op": op, "reqs": _log_int(rng, 1, 512), "newest": _log_int(rng, 1, 2000), "fewest": rng.choice([0, 1]),
            "cached": _log_int(rng, 1, 30000), "page": rng.choice([1, 16, 48, 64, 256]), "lens_seed": seed}


def _lens(case, count, shortest, longest):
    """Lengths of a case, the longest among them."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(shortest, longest) for _ in range(count)]
    lens[r.randrange(count)] = longest
    return lens


def _seq_lens(case):
    return _lens(case, case["seqs"], case["shortest"], case["longest"])


def _kv_lens(case):
    return [max(n, case["steps"]) for n in _lens(case, case["reqs"], case["shortest"], case["longest"])]


def _step_lens(case):
    """(tokens cached, new tokens) of every request of a tables case: most requests decode, some bring a prompt."""
    r = random.Random(case["lens_seed"])
    old = [r.randint(0, case["cached"]) for _ in range(case["reqs"])]
    new = [r.randint(case["fewest"], 1) if r.random() < 0.8 else r.randint(case["fewest"], case["newest"])
           for _ in range(case["reqs"])]
    new[r.randrange(case["reqs"])] = case["newest"]
    return old, new


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "gdn_prefill":
        lens = _seq_lens(case)
        t, hk, hv = sum(lens), case["hk"], case["hv"]
        states = len(lens) * hv * D * D * 4 * (2 if case["initial"] else 1)
        return {"bytes": t * (4 * hk * D + 4 * hv * D + 4 * hv) + states, "flops": t * hv * 6 * D * D}
    if op in ("gdn_decode", "gdn_verify"):
        b, t, hk, hv = case["reqs"], case.get("steps", 1), case["hk"], case["hv"]
        return {"bytes": b * t * (4 * hk * D + 4 * hv * D + 4 * hv) + b * hv * D * D * 4 * (1 + t),
                "flops": b * t * hv * 6 * D * D}
    if op == "paged":
        lens = _kv_lens(case)
        b, t, hq, hk = case["reqs"], case["steps"], case["hq"], case["hk"]
        pages = sum(_pages(n, case["page"]) for n in lens)
        pairs = sum(t * n - t * (t - 1) // 2 for n in lens)
        return {"bytes": sum(lens) * hk * D * 4 + b * t * hq * (D * 4 + 4) + 4 * pages + 4 * b,
                "flops": pairs * hq * 4 * D}
    old, new = _step_lens(case)
    grown = sum(_pages(o + n, case["page"]) - _pages(o, case["page"]) for o, n in zip(old, new))
    touched = sum(_pages(o + n, case["page"]) - o // case["page"] for o, n in zip(old, new))
    return {"bytes": 12 * len(old) + 4 * touched + 8 * grown + sum(new) * 12 + 8, "flops": 4 * sum(new)}


# ---------------------------------------------------------------- inputs
def _gdn_inputs(gen, tokens, hk, hv):
    """Token tensors as a layer's short convolutions and projections leave them: q, k, v = SiLU of normal draws."""
    dev = "cuda"

    def act(h):
        x = torch.randn((tokens, h, D), generator=gen, device=dev)
        return (x * torch.sigmoid(x)).to(torch.bfloat16)

    q, k, v = act(hk), act(hk), act(hv)
    a = torch.randn((tokens, hv), generator=gen, device=dev).to(torch.bfloat16)
    beta = torch.randn((tokens, hv), generator=gen, device=dev).to(torch.bfloat16)
    # decay rates exp(A_log) in [1, 16], softplus(dt_bias) log-uniform in [1e-3, 0.1]
    A_log = torch.log(1 + 15 * torch.rand(hv, generator=gen, device=dev))
    dt = torch.exp(torch.rand(hv, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    dt_bias = dt + torch.log(-torch.expm1(-dt))
    return {"q": q, "k": k, "v": v, "a": a, "beta": beta, "A_log": A_log, "dt_bias": dt_bias}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "gdn_prefill":
        lens = _seq_lens(case)
        hv = case["hv"]
        s.update(_gdn_inputs(gen, sum(lens), case["hk"], hv))
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        s["cu_host"] = torch.from_numpy(cu)
        s["cu"] = s["cu_host"].cuda()
        s["pool"] = s["slots"] = None
        if case["initial"]:
            s["pool"] = 0.05 * torch.randn((len(lens) + 3, hv, D, D), generator=gen, device="cuda")
            s["slots"] = torch.randperm(len(lens) + 3, generator=gen, device="cuda")[:len(lens)].to(torch.int32)
        # what a serving program keeps: output, states and the workspace of the call
        s["out"] = torch.empty_like(s["v"])
        s["final"] = torch.empty((len(lens), hv, D, D), dtype=torch.float32, device="cuda")
        if own:
            import kda_linear_attention_bounded_gb300 as kda
            s["ws"] = kda.make_workspace(nbytes=kda.gdn_prefill_workspace_size(sum(lens), len(lens), hv))
    elif op in ("gdn_decode", "gdn_verify"):
        b, t, hv = case["reqs"], case.get("steps", 1), case["hv"]
        s.update(_gdn_inputs(gen, b * t, case["hk"], hv))
        s["pool"] = 0.05 * torch.randn((case["slots"], hv, D, D), generator=gen, device="cuda")
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:b].to(torch.int32)
        s["out"] = torch.empty_like(s["v"])
        if op == "gdn_verify":
            s["inter"] = torch.empty((b, t, hv, D, D), dtype=torch.float32, device="cuda")
        if own:
            import kda_linear_attention_bounded_gb300 as kda
            s["ws"] = kda.make_workspace()
    elif op == "paged":
        lens, b, t, hq, hk, page = (_kv_lens(case), case["reqs"], case["steps"], case["hq"], case["hk"], case["page"])
        pages = [_pages(n, page) for n in lens]
        total, width = sum(pages), max(pages)
        s["k_pages"] = torch.randn((total + 2, page, hk, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["v_pages"] = torch.randn((total + 2, page, hk, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["q"] = 1.5 * torch.randn((b * t, hq, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        # pages in the order a long-running allocator hands them out: any
        order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        n_pages = torch.tensor(pages, device="cuda")
        first = torch.cumsum(n_pages, 0) - n_pages
        col = torch.arange(width, device="cuda")
        at = (first[:, None] + col).clamp(max=total - 1)
        s["table"] = torch.where(col < n_pages[:, None], order[at], torch.zeros_like(order[at])).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b * t, hq), dtype=torch.float32, device="cuda")
        if own:
            import kda_linear_attention_bounded_gb300 as kda
            s["ws"] = kda.make_workspace(nbytes=kda.paged_workspace_size(hq, hk, t))
    else:
        old, new = _step_lens(case)
        page, b = case["page"], case["reqs"]
        most = max(_pages(o + n, page) for o, n in zip(old, new))
        total = sum(_pages(o + n, page) for o, n in zip(old, new))
        order = torch.randperm(total + 5, generator=gen, device="cuda").to(torch.int32)
        had = torch.tensor([_pages(o, page) for o in old], device="cuda")
        first = torch.cumsum(had, 0) - had
        col = torch.arange(most, device="cuda")
        at = (first[:, None] + col).clamp(max=total - 1)
        s["table"] = torch.where(col < had[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
        s["free"] = order[sum(_pages(o, page) for o in old):].contiguous()
        s["old"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        # a captured step has room for a bucket of tokens, more than this step brings
        room = sum(new) + 7
        for name, n, dt in (("cu", b + 1, torch.int32), ("kv_lens", b, torch.int32), ("positions", room, torch.int32),
                            ("slot_map", room, torch.int64), ("used", 1, torch.int32)):
            s[name] = torch.zeros(n, dtype=dt, device="cuda")
        if own:
            import kda_linear_attention_bounded_gb300 as kda
            s["ws"] = kda.make_workspace()
    return s


# ---------------------------------------------------------------- plain forms
def _unit_norm(x):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _log_decay(a, A_log, dt_bias):
    x = a.float() + dt_bias
    return -torch.exp(A_log) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))


def _unit_lower_inverse(L):
    """Inverse of I + A for strictly lower A ([..., n, n], n a power of two): blocks of twice the size each turn,
    [[X1, 0], [-X2 A21 X1, X2]]."""
    n = L.shape[-1]
    X = torch.eye(n, device=L.device, dtype=L.dtype).expand(L.shape).clone()
    size = 1
    while size < n:
        blocks = L.reshape(*L.shape[:-2], n // (2 * size), 2 * size, n // (2 * size), 2 * size)
        inv = X.reshape(*L.shape[:-2], n // (2 * size), 2 * size, n // (2 * size), 2 * size)
        A21 = torch.diagonal(blocks[..., size:, :, :size], dim1=-4, dim2=-2).movedim(-1, -3)
        X1 = torch.diagonal(inv[..., :size, :, :size], dim1=-4, dim2=-2).movedim(-1, -3)
        X2 = torch.diagonal(inv[..., size:, :, size:], dim1=-4, dim2=-2).movedim(-1, -3)
        X21 = -(X2 @ A21 @ X1)
        torch.diagonal(inv[..., size:, :, :size], dim1=-4, dim2=-2).movedim(-1, -3).copy_(X21)
        size *= 2
    return X


def _plain_gdn_prefill(s):
    """The chunked form: every chunk of 64 tokens at once for what does not depend on the state, then the states
    chunk by chunk (the sequences that still have one, longest first)."""
    hk, hv = s["case"]["hk"], s["case"]["hv"]
    dev = s["q"].device
    cu = s["cu_host"].tolist()
    lens = [y - x for x, y in zip(cu, cu[1:])]
    by_len = sorted(range(len(lens)), key=lambda n: -lens[n])
    count = [_pages(lens[n], CHUNK) for n in by_len]
    first = [sum(count[:i]) for i in range(len(count))]
    starts = torch.tensor([cu[n] + j * CHUNK for n, c in zip(by_len, count) for j in range(c)], device=dev)
    ends = torch.tensor([cu[n + 1] for n, c in zip(by_len, count) for _ in range(c)], device=dev)
    token = starts[:, None] + torch.arange(CHUNK, device=dev)
    live = token < ends[:, None]                                  # [chunks, 64]
    token = token.clamp(max=cu[-1] - 1)
    group = hv // hk

    def rows(x):   # [tokens, H, ...] -> [chunks, H, 64, ...]
        return x[token].transpose(1, 2)

    m = live[:, None, :, None]
    q = (rows(_unit_norm(s["q"])) * m).repeat_interleave(group, 1)
    k = (rows(_unit_norm(s["k"])) * m).repeat_interleave(group, 1)
    v = rows(s["v"].float()) * m
    beta = rows(torch.sigmoid(s["beta"].float())) * live[:, None]
    lam = rows(_log_decay(s["a"], s["A_log"], s["dt_bias"])) * live[:, None]
    b = torch.cumsum(lam.double(), -1)
    end = b[..., -1:]
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=dev).tril()
    decay = torch.where(lower, torch.exp(torch.where(lower, b[..., :, None] - b[..., None, :], 0.0)), 0.0).float()
    A = torch.tril((k @ k.mT) * decay, -1) * beta[..., None]
    X = _unit_lower_inverse(A)
    eb = torch.exp(b).float()[..., None]
    u0 = X @ (v * beta[..., None])
    w = X @ (k * (beta[..., None] * eb))
    P = (q @ k.mT) * decay * SCALE
    q_in = q * (eb * SCALE)
    k_out = k * torch.exp(end - b).float()[..., None]
    gamma = torch.exp(end).float()[..., None]
    S = torch.zeros((len(lens), hv, D, D), device=dev)
    order = torch.tensor(by_len, device=dev)
    if s["pool"] is not None:
        S = s["pool"][s["slots"].long()[order]]
    o = torch.empty_like(v)
    first_t = torch.tensor(first, device=dev)
    for j in range(count[0]):                                     # the recurrence over chunks
        n = sum(c > j for c in count)
        at = first_t[:n] + j
        U = u0[at] - w[at] @ S[:n]
        o[at] = q_in[at] @ S[:n] + P[at] @ U
        S[:n] = gamma[at] * S[:n] + k_out[at].mT @ U
    out, final = s["out"], s["final"]
    out[token[live]] = o.transpose(1, 2)[live].to(out.dtype)
    final[order] = S
    return out, final


def _plain_gdn_steps(s, update_pool):
    """Token by token from the pool's states: verify records every state, decode puts the last one back."""
    hk, hv = s["case"]["hk"], s["case"]["hv"]
    b, steps = s["case"]["reqs"], s["case"].get("steps", 1)
    group = hv // hk
    q = _unit_norm(s["q"]).repeat_interleave(group, 1).view(b, steps, hv, D)
    k = _unit_norm(s["k"]).repeat_interleave(group, 1).view(b, steps, hv, D)
    v = s["v"].float().view(b, steps, hv, D)
    beta = torch.sigmoid(s["beta"].float()).view(b, steps, hv, 1)
    alpha = torch.exp(_log_decay(s["a"], s["A_log"], s["dt_bias"])).view(b, steps, hv, 1, 1)
    S = s["pool"][s["slots"].long()]
    out = s["out"].view(b, steps, hv, D)
    for t in range(steps):                                        # the recurrence over tokens
        S = alpha[:, t] * S
        u = beta[:, t] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = (SCALE * (S * q[:, t, :, :, None]).sum(-2)).to(out.dtype)
        if not update_pool:
            s["inter"][:, t] = S
    if not update_pool:
        return s["out"], s["inter"]
    s["pool"][s["slots"].long()] = S
    return s["out"], s["pool"]


def _plain_paged(s):
    """Every request's keys and values gathered to the longest length, scores masked behind each row's last token."""
    b, t, hq, hk, page = (s["case"][n] for n in ("reqs", "steps", "hq", "hk", "page"))
    group, width = hq // hk, s["table"].shape[1]
    pages = s["table"].long()
    k = s["k_pages"][pages].view(b, width * page, hk, D).permute(0, 2, 3, 1).float()     # [b, hk, D, n]
    q = s["q"].float().view(b, t, hk, group, D).permute(0, 2, 1, 3, 4).reshape(b, hk, t * group, D)
    score = (q @ k) * SCALE
    del k
    last = s["lens"].long()[:, None] - t + torch.arange(t, device=q.device)              # last visible token of a row
    seen = torch.arange(width * page, device=q.device) <= last[..., None]                # [b, t, n]
    seen = seen[:, None, :, None].expand(b, 1, t, group, width * page).reshape(b, 1, t * group, -1)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_pages"][pages].view(b, width * page, hk, D).permute(0, 2, 1, 3).float()
    o = (p @ v) / total

    def rows(x):   # [b, hk, t group, n] -> [b t, hq, n]
        return x.view(b, hk, t, group, -1).permute(0, 2, 1, 3, 4).reshape(b * t, hq, -1)

    s["out"].copy_(rows(o))
    s["lse"].copy_(rows(top + torch.log(total))[..., 0])
    return s["out"], s["lse"]


def _plain_tables(s):
    page = s["case"]["page"]
    old, new, table = s["old"].long(), s["new"].long(), s["table"]
    cu = torch.cumsum(new, 0)
    start = cu - new
    had, has = (old + page - 1) // page, (old + new + page - 1) // page
    grown = has - had
    taken = torch.cumsum(grown, 0) - grown
    s["cu"][0] = 0
    s["cu"][1:] = cu.to(torch.int32)
    s["kv_lens"].copy_(old + new)
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= had[:, None]) & (col < has[:, None])
    pick = (taken[:, None] + col - had[:, None]).clamp(0, s["free"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free"][pick], table))
    tok = torch.arange(s["slot_map"].shape[0], device=table.device)
    req = (tok[:, None] >= cu[None, :]).sum(-1)
    live = req < old.shape[0]
    req = req.clamp(max=old.shape[0] - 1)
    pos = old[req] + tok - start[req]
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slot_map"].copy_(torch.where(live, slot, -1))
    s["used"].copy_(grown.sum())
    return table, s["cu"], s["kv_lens"], s["positions"], s["slot_map"], s["used"]


# ---------------------------------------------------------------- the framework's calls
def _own_run(s):
    import kda_linear_attention_bounded_gb300 as kda

    op = s["op"]
    if op == "gdn_prefill":
        return kda.gdn_chunk_prefill(s["q"], s["k"], s["v"], s["a"], s["beta"], s["A_log"], s["dt_bias"], s["cu"],
                                     s["cu_host"], state_pool=s["pool"], slot_ids=s["slots"],
                                     load_initial=s["pool"] is not None, out=s["out"], final_state=s["final"],
                                     workspace=s["ws"])
    if op == "gdn_verify":
        return kda.gdn_recurrent_verify(s["q"], s["k"], s["v"], s["a"], s["beta"], s["A_log"], s["dt_bias"],
                                        s["pool"], s["slots"], s["case"]["steps"], out=s["out"],
                                        intermediate_states=s["inter"], workspace=s["ws"])
    if op == "gdn_decode":
        out = kda.gdn_decode(s["q"], s["k"], s["v"], s["a"], s["beta"], s["A_log"], s["dt_bias"], s["pool"],
                             s["slots"], out=s["out"], workspace=s["ws"])
        return out, s["pool"]
    if op == "paged":
        return kda.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["case"]["steps"],
                                   out=s["out"], lse=s["lse"], workspace=s["ws"])
    kda.step_tables(s["table"], s["old"], s["new"], s["free"], s["case"]["page"], cu_seqlens=s["cu"],
                    kv_lens=s["kv_lens"], positions=s["positions"], slot_map=s["slot_map"], pages_used=s["used"],
                    workspace=s["ws"])
    return s["table"], s["cu"], s["kv_lens"], s["positions"], s["slot_map"], s["used"]


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "gdn_prefill":
        return _plain_gdn_prefill(state)
    if op in ("gdn_decode", "gdn_verify"):
        return _plain_gdn_steps(state, op == "gdn_decode")
    return _plain_paged(state) if op == "paged" else _plain_tables(state)


# ---------------------------------------------------------------- 64-bit definitions
def _exact_recurrence(s, sequences, S):
    """The recurrence token by token in fp64; ``sequences``: lists of token rows, longest first; S: [n, hv, D, D].
    Yields the states after every step with the sequences still running."""
    hk, hv = s["case"]["hk"], s["case"]["hv"]
    dev = s["q"].device
    head = torch.arange(hv, device=dev) // (hv // hk)
    A, bias = torch.exp(s["A_log"].double()), s["dt_bias"].double()
    out = torch.zeros((s["q"].shape[0], hv, D), dtype=torch.float64, device=dev)
    length = max(len(x) for x in sequences)
    grid = torch.tensor([list(x) + [0] * (length - len(x)) for x in sequences], device=dev)
    running = [0] * (length + 1)
    for x in sequences:
        running[len(x)] += 1
    n = len(sequences)
    for t in range(length):
        n -= running[t]
        rows = grid[:n, t]
        q, k, v = s["q"][rows].double(), s["k"][rows].double(), s["v"][rows].double()
        q = (q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6))[:, head]
        k = (k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6))[:, head]
        beta = 1 / (1 + torch.exp(-s["beta"][rows].double()))
        alpha = torch.exp(-A * torch.logaddexp(s["a"][rows].double() + bias, torch.zeros((), dtype=torch.float64, device=dev)))
        S[:n] *= alpha[..., None, None]
        err = beta[..., None] * (v - (k[:, :, None, :] @ S[:n])[:, :, 0])
        S[:n] += k[..., None] * err[:, :, None, :]
        out[rows] = SCALE * (q[:, :, None, :] @ S[:n])[:, :, 0]
        yield t, n, S, out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gdn_prefill":
        cu = s["cu_host"].tolist()
        order = sorted(range(len(cu) - 1), key=lambda n: cu[n] - cu[n + 1])
        S = torch.zeros((len(order), case["hv"], D, D), dtype=torch.float64, device="cuda")
        if s["pool"] is not None:
            S = s["pool"][s["slots"].long()].double()[order]
        for _, _, S, out in _exact_recurrence(s, [range(cu[n], cu[n + 1]) for n in order], S):
            pass
        final = torch.empty_like(S)
        final[order] = S
        return out, final
    if op in ("gdn_decode", "gdn_verify"):
        b, steps = case["reqs"], case.get("steps", 1)
        S = s["pool"][s["slots"].long()].double()
        inter = []
        for _, _, S, out in _exact_recurrence(s, [range(i * steps, (i + 1) * steps) for i in range(b)], S):
            if op == "gdn_verify":
                inter.append(S.clone())
        if op == "gdn_verify":
            return out, torch.stack(inter, 1)
        pool = s["pool"].double()
        pool[s["slots"].long()] = S
        return out, pool
    if op == "paged":
        t, hq, hk, page = case["steps"], case["hq"], case["hk"], case["page"]
        out = torch.empty((s["q"].shape[0], hq, D), dtype=torch.float64, device="cuda")
        lse = torch.empty((s["q"].shape[0], hq), dtype=torch.float64, device="cuda")
        for i, n in enumerate(_kv_lens(case)):
            pos = torch.arange(n, device="cuda")
            at = s["table"][i].long()[pos // page]
            k, v = s["k_pages"][at, pos % page], s["v_pages"][at, pos % page]
            for h in range(hk):
                mine = slice(h * (hq // hk), (h + 1) * (hq // hk))
                kh, vh = k[:, h].double(), v[:, h].double()
                for j in range(t):
                    last = n - t + j + 1
                    z = s["q"][i * t + j, mine].double() @ kh[:last].T / math.sqrt(D)
                    lse[i * t + j, mine] = torch.logsumexp(z, -1)
                    out[i * t + j, mine] = torch.softmax(z, -1) @ vh[:last]
        return out, lse
    return None
