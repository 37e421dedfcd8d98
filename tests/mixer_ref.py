"""Plain 64-bit implementations of the mixers beside KDA for the tests: token by token, row by row, pair by pair. They
share no code with the package."""
import torch

from tests.block_ref import spans

F64 = torch.float64


def gdn(q, k, v, a, beta, scale, A_log, dt_bias, init, cu=None, l2=False):
    """q, k [B, T, HK, D], v [B, T, H, D], a, beta [B, T, H]; returns out [B, T, H, D] and states [S, H, D, D] ([v][k])."""
    B, T, H, D = v.shape
    q, k, v, a, beta = (t.double().reshape(B * T, *t.shape[2:]) for t in (q, k, v, a, beta))
    if l2:
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    q, k = (t.repeat_interleave(H // t.shape[1], 1) for t in (q, k))
    u = a if dt_bias is None else a + dt_bias.double()
    keep = torch.exp(-torch.exp(A_log.double()) * torch.nn.functional.softplus(u, threshold=200.0))
    b, out, fins = torch.sigmoid(beta), torch.zeros_like(v), []
    for i, (s0, s1) in enumerate(spans(B, T, cu)):
        S = init[i].double().clone() if init is not None else v.new_zeros(H, D, D)
        for t in range(s0, s1):
            S = keep[t][:, None, None] * S
            miss = b[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
            S = S + miss[:, :, None] * k[t][:, None]
            out[t] = scale * torch.einsum("hvk,hk->hv", S, q[t])
        fins.append(S)
    return out.view(B, T, H, D), torch.stack(fins)


def rope(x, weight, positions, inv_freq, norm, interleaved, eps):
    """x [..., heads, D]; returns the turned heads and, per element, the sum of |terms| of it."""
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    y, mag = x.clone(), x.abs()
    half = 0 if inv_freq is None else inv_freq.numel()
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        t = (positions.double() * inv_freq[p].double())[..., None]
        c, s = torch.cos(t), torch.sin(t)
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
        mag[..., i] = mag[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, mag


def attn_step(q, k_cache, v_cache, table, positions, scale):
    """q [S, H, D], caches [pages, HK, page, D]; returns out, lse, the weights' sum of |p v| and the scores' size."""
    S, H, D = q.shape
    HK, page = k_cache.shape[1:3]
    out, mag = torch.zeros(S, H, D, dtype=F64, device=q.device), torch.zeros(S, H, D, dtype=F64, device=q.device)
    lse, size = torch.full((S, H), -torch.inf, dtype=F64, device=q.device), torch.zeros(S, H, dtype=F64, device=q.device)
    for s in range(S):
        n = int(positions[s]) + 1
        if n <= 0:
            continue
        pages = table[s, :(n + page - 1) // page].long()
        for h in range(H):
            k, v = (c[pages, h // (H // HK)].reshape(-1, D)[:n].double() for c in (k_cache, v_cache))
            x = scale * (k @ q[s, h].double())
            p = torch.softmax(x, 0)
            out[s, h], mag[s, h], lse[s, h] = p @ v, p @ v.abs(), torch.logsumexp(x, 0)
            size[s, h] = (abs(scale) * (k.abs() @ q[s, h].double().abs())).max()
    return out, lse, mag, size
