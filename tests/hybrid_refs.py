"""Plain 64-bit forms of the gated delta rule, paged attention and the step tables (torch, CPU)."""
import math

import torch

D = 128


def gdn_inputs(tokens, hk, hv, seed, a_mean=0.0, device="cuda"):
    """q, k, v = SiLU of normal draws, a and beta_logits normal (bf16); decay rates in [1, 16], softplus(dt_bias)
    log-uniform in [1e-3, 0.1]."""
    g = torch.Generator().manual_seed(seed)
    act = lambda h: torch.nn.functional.silu(torch.randn((tokens, h, D), generator=g)).bfloat16().to(device)  # noqa: E731
    q, k, v = act(hk), act(hk), act(hv)
    a = (torch.randn((tokens, hv), generator=g) + a_mean).bfloat16().to(device)
    beta = torch.randn((tokens, hv), generator=g).bfloat16().to(device)
    A_log = torch.log(1 + 15 * torch.rand(hv, generator=g)).to(device)
    dt = torch.exp(torch.rand(hv, generator=g) * math.log(100.0) + math.log(1e-3))
    return [q, k, v, a, beta, A_log, (dt + torch.log(-torch.expm1(-dt))).to(device)]


def gdn_reference(x, lens, S0=None, scale=D ** -0.5, keep=True):
    """(out [tokens, Hv, D], states after every token: list per sequence of [len, Hv, D, D] if keep, final [N, Hv, D, D])."""
    q, k, v, a, beta, A_log, dt_bias = (t.detach().double().cpu() for t in x)
    hv = v.shape[1]
    group = hv // q.shape[1]
    q = (q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(group, 1)
    k = (k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(group, 1)
    lam = -torch.exp(A_log) * torch.logaddexp(a + dt_bias, torch.zeros((), dtype=torch.float64))
    alpha, beta = torch.exp(lam), torch.sigmoid(beta)
    out = torch.zeros((q.shape[0], hv, D), dtype=torch.float64)
    steps, final, t = [], [], 0
    for n, length in enumerate(lens):
        S = torch.zeros((hv, D, D), dtype=torch.float64) if S0 is None else S0[n].double().cpu().clone()
        rec = []
        for _ in range(length):
            S = alpha[t][:, None, None] * S
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            out[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
            if keep:
                rec.append(S)
            t += 1
        steps.append(torch.stack(rec) if rec else torch.zeros((0, hv, D, D), dtype=torch.float64))
        final.append(S)
    return out, steps, torch.stack(final)


def rel_l2(x, ref):
    x, ref = x.detach().double().cpu(), ref.double().cpu()
    den = ref.norm()
    return float((x - ref).norm() / den) if den > 0 else float((x - ref).norm())


def paged_reference(q, k_pages, v_pages, table, lens, T, scale=D ** -0.5):
    """(out [B*T, Hq, D], lse [B*T, Hq]) in fp64: request by request, row by row."""
    q, k_pages, v_pages = (t.detach().double().cpu() for t in (q, k_pages, v_pages))
    table, page, hk = table.cpu(), k_pages.shape[1], k_pages.shape[2]
    hq = q.shape[1]
    out = torch.zeros((q.shape[0], hq, D), dtype=torch.float64)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        pos = torch.arange(max(n, 0))
        at = table[b].long()[pos // page] if n > 0 else pos
        k, v = k_pages[at, pos % page], v_pages[at, pos % page]
        for t in range(T):
            seen = n - T + t + 1
            if seen <= 0:
                continue
            for h in range(hk):
                mine = slice(h * (hq // hk), (h + 1) * (hq // hk))
                z = scale * (q[b * T + t, mine] @ k[:seen, h].T)
                lse[b * T + t, mine] = torch.logsumexp(z, -1)
                out[b * T + t, mine] = torch.softmax(z, -1) @ v[:seen, h]
    return out, lse
