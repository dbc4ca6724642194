"""The chunked gated delta rule in 64 bits with its operands rounded as the kernels round them, or otherwise (torch, CPU):
what a rounding costs a final state."""
import torch

from hybrid_refs import D


def pair(x, t):
    """x as the sum of two values of type t."""
    hi = x.to(t).double()
    return hi + (x - hi).to(t).double()


def final_states(x, lens, of_s=None, of_others=None, S0=None):
    """Final states [N, Hv, D, D] with S as a pair of `of_s` where it meets the keys and L, R and U as pairs of `of_others`
    (each value channel times a power of two that fp16 holds); None: not rounded."""
    q, k, v, a, beta, A_log, dt_bias = (t.detach().double().cpu() for t in x)
    k = (k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(v.shape[1] // q.shape[1], 1)
    lam = -torch.exp(A_log) * torch.logaddexp(a + dt_bias, torch.zeros((), dtype=torch.float64))
    beta = torch.sigmoid(beta)
    rounded = lambda y, t: y if t is None else pair(y, t)  # noqa: E731
    final, t0 = [], 0
    for n, length in enumerate(lens):
        S = torch.zeros((v.shape[1], D, D), dtype=torch.float64) if S0 is None else S0[n].double().cpu()
        for c in range(t0, t0 + length, 64):
            e = min(c + 64, t0 + length)
            K, V, B, b = k[c:e].transpose(0, 1), v[c:e].transpose(0, 1), beta[c:e].T, lam[c:e].T.cumsum(-1)
            A = torch.tril(B[:, :, None] * (K @ K.mT) * torch.exp((b[:, :, None] - b[:, None, :]).clamp(max=0)), -1)
            L = torch.linalg.inv(torch.eye(e - c, dtype=torch.float64) + A)
            R = B[:, :, None] * (V - torch.exp(b)[:, :, None] * (K @ rounded(S, of_s)))
            size = 2.0 ** torch.floor(torch.log2(2.0 ** 8 / R.abs().amax(1, keepdim=True).clamp(min=1e-30)))
            U = rounded(L, of_others) @ rounded(R * size, of_others)
            end = torch.exp(b[:, -1:] - b)[:, :, None]
            S = torch.exp(b[:, -1])[:, None, None] * S + K.mT @ (rounded(end * U, of_others) / size)
        final.append(S)
        t0 += length
    return torch.stack(final)
