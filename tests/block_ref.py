"""Plain 64-bit implementations of the operators around the mixer, token by token, for the tests.
They share no code with the package. Each also returns what bounds the rounding of a result: the
same sums taken over absolute values."""
import torch

F64 = torch.float64


def spans(B, T, cu):
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    cu = [int(v) for v in cu]
    return list(zip(cu[:-1], cu[1:]))


def act(z, name):
    return z * torch.sigmoid(z) if name == "silu" else torch.sigmoid(z) if name == "sigmoid" else z


def conv(x, weight, bias, silu, init, cu=None):
    """x [B, T, C]; returns out, final rows [S, W - 1, C], and the sum of |terms| of every output."""
    B, T, C = x.shape
    W = weight.shape[1]
    flat, w = x.double().reshape(B * T, C), weight.double()
    out, mag = torch.zeros_like(flat), torch.zeros_like(flat)
    fins = []
    for i, (b, e) in enumerate(spans(B, T, cu)):
        first = init[i].double() if init is not None else flat.new_zeros(W - 1, C)
        ext = torch.cat([first, flat[b:e]])
        u = torch.zeros(e - b, C, dtype=F64, device=x.device)
        m = torch.zeros_like(u)
        for j in range(W):
            u += ext[j:j + e - b] * w[:, j]
            m += (ext[j:j + e - b] * w[:, j]).abs()
        if bias is not None:
            u += bias.double()
            m += bias.double().abs()
        out[b:e], mag[b:e] = (act(u, "silu") if silu else u), m
        fins.append(ext[e - b:])
    return out.view(B, T, C), torch.stack(fins), mag.view(B, T, C)


def ssm(x, dt, b, c, A_log, D, dt_bias, init, cu=None):
    """x [B, T, H, P], dt [B, T, H], b and c [B, T, G, N]; returns out, states, and both with every
    term replaced by its absolute value."""
    B, T, H, P = x.shape
    G, N = b.shape[2:]
    x, dt, b, c = (v.double().reshape(B * T, *v.shape[2:]) for v in (x, dt, b, c))
    b, c = (v.repeat_interleave(H // G, 1) for v in (b, c))
    if dt_bias is not None:
        dt = dt + dt_bias.double()
    delta = torch.nn.functional.softplus(dt, threshold=200.0)
    keep = torch.exp(-torch.exp(A_log.double()) * delta)
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    fins, mags = [], []
    for i, (s0, s1) in enumerate(spans(B, T, cu)):
        S = init[i].double().clone() if init is not None else x.new_zeros(H, P, N)
        M = S.abs()
        for t in range(s0, s1):
            k = keep[t][:, None, None]
            S = k * S + (delta[t][:, None] * x[t])[:, :, None] * b[t][:, None]
            M = k * M + (delta[t][:, None] * x[t].abs())[:, :, None] * b[t][:, None].abs()
            out[t] = (S * c[t][:, None]).sum(-1)
            mag[t] = (M * c[t][:, None].abs()).sum(-1)
        fins.append(S)
        mags.append(M)
    if D is not None:
        out += D.double()[:, None] * x
        mag += (D.double()[:, None] * x).abs()
    return out.view(B, T, H, P), torch.stack(fins), mag.view(B, T, H, P), torch.stack(mags)


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm(x, gate, weight, name, gate_first, eps):
    x, z = x.double(), act(gate.double(), name)
    n = rms(x * z, eps) if gate_first else rms(x, eps) * z
    return n if weight is None else n * weight.double()


def residual_norm(x, residual, weight, post, gate, name, chan, alpha, eps):
    u = x.double()
    if post is not None:
        u = rms(u, eps) * post.double()
    if gate is not None:
        u = u * act(gate.double(), name)
    if chan is not None:
        u = u * chan.double()
    r = residual.double() + alpha * u
    n = rms(r, eps)
    return (n if weight is None else n * weight.double()), r, residual.double().abs() + (alpha * u).abs()
