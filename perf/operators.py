"""Measured cases of the operators around a recurrent mixer: short causal convolution (``conv``), selective
state-space scan (``ssm``), gated norm (``gated_norm``) and residual norm (``residual_norm``), each for prompts and
for single tokens. ``run`` computes a case with elementary torch operations (``own`` false) or with this framework's
calls (``own`` true); ``exact`` is the definition in 64 bits, token by token.

Sizes are the framework's own workloads (8 x 4096 tokens of 16 heads, 16 packed sequences of 32 heads, one
131072-token sequence of 32 heads, 128-sequence decode) with heads of 128 or 64 channels and a state of 128.
"""
import math

import torch

own = False

N = 128           # state channels of the scan
CHUNK = 128       # tokens per chunk of the plain scan
EPS = 1e-5


def listed():
    return [
        # one of the q / k / v convolutions of a 16-head layer, read out of the packed projection
        {"name": "conv_b8_t4096_c2048", "op": "conv", "B": 8, "T": 4096, "C": 2048, "W": 4, "extra": 4096, "varlen": 0,
         "states": False, "silu": True},
        # the x|B|C convolution of a 32-head scan layer over packed prompts, with the states of a chunked prefill
        {"name": "conv_varlen16_c4352", "op": "conv", "B": 1, "T": 65519, "C": 4352, "W": 4, "extra": 0, "varlen": 16,
         "states": True, "silu": True},
        # one decoding step of 128 sequences
        {"name": "conv_step_s128_c6144", "op": "conv_step", "S": 128, "C": 6144, "W": 4, "silu": True},
        # a batch of prompts
        {"name": "ssm_b8_t4096_h16", "op": "ssm", "B": 8, "T": 4096, "H": 16, "P": 128, "G": 1, "varlen": 0,
         "init": False, "state": "fp32"},
        # packed prompts of ragged lengths, small heads in groups, states carried from an earlier call
        {"name": "ssm_varlen16_h32_p64", "op": "ssm", "B": 1, "T": 65519, "H": 32, "P": 64, "G": 4, "varlen": 16,
         "init": True, "state": "bf16"},
        # one long document: few states, a long chain
        {"name": "ssm_b1_t131072_h32", "op": "ssm", "B": 1, "T": 131072, "H": 32, "P": 128, "G": 1, "varlen": 0,
         "init": True, "state": "fp32"},
        # a short prompt of one user, where latency counts
        {"name": "ssm_b1_t53_h8_p64", "op": "ssm", "B": 1, "T": 53, "H": 8, "P": 64, "G": 1, "varlen": 0,
         "init": True, "state": "fp32"},
        # one decoding step of 128 sequences
        {"name": "ssm_step_s128_h16", "op": "ssm_step", "S": 128, "H": 16, "P": 128, "G": 1, "state": "fp32"},
        # the head-wise norm after a 16-head mixer with its sigmoid gate
        {"name": "gated_norm_t32768_h16", "op": "gated_norm", "T": 32768, "R": 16, "D": 128, "act": "sigmoid",
         "gate_first": False, "extra": 0},
        # the norm over a scan layer's whole row, gate first, for one decoding step; the gate is a projection's slice
        {"name": "gated_norm_s128_d2048", "op": "gated_norm", "T": 128, "R": 1, "D": 2048, "act": "silu",
         "gate_first": True, "extra": 4352},
        # between two blocks of a 16-head model, prompts
        {"name": "residual_norm_t32768_d2048", "op": "residual_norm", "T": 32768, "D": 2048, "residual": "bf16",
         "post": False, "gate": "", "chan": False, "alpha": 1.0},
        # the same with a norm after the block, its gate and a learned scale on a 32-bit stream, a few sequences' step
        {"name": "residual_norm_s8_d4096", "op": "residual_norm", "T": 8, "D": 4096, "residual": "fp32",
         "post": True, "gate": "sigmoid", "chan": True, "alpha": 0.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_step", "ssm", "ssm", "ssm", "ssm_step", "gated_norm", "residual_norm"])
    if op == "conv":
        C, W, varlen = 8 * _log_int(rng, 1, 544), rng.choice([2, 3, 4]), rng.choice([0, 0, rng.randint(2, 24)])
        T = _log_int(rng, 1, min(131072, (1 << 28) // C))
        B = 1 if varlen else _log_int(rng, 1, max(1, min(16, (1 << 28) // (C * T))))
        return {"op": op, "B": B, "T": max(T, varlen), "C": C, "W": W, "extra": rng.choice([0, 8 * rng.randint(1, 64)]),
                "varlen": varlen, "states": rng.random() < 0.6, "silu": rng.random() < 0.8}
    if op == "conv_step":
        return {"op": op, "S": _log_int(rng, 1, 256), "C": 8 * _log_int(rng, 1, 1024), "W": rng.choice([2, 3, 4]),
                "silu": rng.random() < 0.8}
    if op in ("ssm", "ssm_step"):
        G = rng.choice([1, 1, 2, 4])
        H, P = G * _log_int(rng, 1, 32 // G), rng.choice([64, 128])
        base = {"op": op, "H": H, "P": P, "G": G, "state": rng.choice(["fp32", "bf16"])}
        if op == "ssm_step":
            return {"S": _log_int(rng, 1, 128), **base}
        varlen = rng.choice([0, 0, rng.randint(2, 24)])
        T = _log_int(rng, 1, min(131072, (1 << 22) // H))
        B = 1 if varlen else _log_int(rng, 1, max(1, min(16, (1 << 22) // (H * T))))
        return {"B": B, "T": max(T, varlen), "varlen": varlen, "init": rng.random() < 0.6, **base}
    if op == "gated_norm":
        D = rng.choice([64, 128, 8 * _log_int(rng, 1, 1024)])
        R = _log_int(rng, 1, max(1, min(32, 4096 // D)))
        return {"op": op, "T": _log_int(rng, 1, min(65536, (1 << 26) // (D * R))), "R": R, "D": D,
                "act": rng.choice(["sigmoid", "silu"]), "gate_first": rng.random() < 0.5,
                "extra": rng.choice([0, 8 * rng.randint(1, 64)])}
    D = 8 * _log_int(rng, 1, 1024)
    return {"op": op, "T": _log_int(rng, 1, min(65536, (1 << 26) // D)), "D": D, "residual": rng.choice(["bf16", "fp32"]),
            "post": rng.random() < 0.5, "gate": rng.choice(["", "sigmoid", "silu"]), "chan": rng.random() < 0.4,
            "alpha": rng.choice([1.0, 0.5])}


_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _lengths(case, seed):
    """`varlen` positive lengths that add up to T, spread as those of a batch of prompts are."""
    n, T = case["varlen"], case["T"]
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=gen).double() + 0.02
    ends = torch.floor(torch.cumsum(w, 0) / w.sum() * (T - n)).long() + torch.arange(1, n + 1)
    ends[-1] = T
    return [int(v) for v in torch.diff(ends, prepend=ends.new_zeros(1))]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    op, s = case["op"], {}
    if op in ("conv", "ssm"):
        s["lengths"], s["cu"] = None, None
        if case["varlen"]:
            s["lengths"] = _lengths(case, seed)
            s["cu"] = torch.tensor([0] + s["lengths"], dtype=torch.int64).cumsum(0).cuda()
        seqs = case["varlen"] or case["B"]
    if op == "conv":
        B, T, C, W = case["B"], case["T"], case["C"], case["W"]
        s["x"] = randn(B, T, C + case["extra"])[:, :, :C]  # the first channels of a wider projection
        s["init"] = randn(seqs, W - 1, C) if case["states"] else None
    if op == "conv_step":
        C, W = case["C"], case["W"]
        s["x"], s["state"] = randn(case["S"], C), randn(case["S"], W - 1, C)
    if op in ("conv", "conv_step"):
        s["weight"], s["bias"] = randn(C, W, dtype=torch.float32, scale=W ** -0.5), randn(C, dtype=torch.float32, scale=0.1)
    if op in ("ssm", "ssm_step"):
        H, P, G = case["H"], case["P"], case["G"]
        tok = (case["B"], case["T"]) if op == "ssm" else (case["S"],)
        # x, B and C are slices of one row of the convolution's output, as a layer has them
        xbc = randn(*tok, H * P + 2 * G * N)
        s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
        s["b"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["c"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
        s["dt"] = randn(*tok, H)
        s["A_log"] = torch.log(1 + 15 * rand(H))
        step = torch.exp(rand(H) * math.log(100.0) + math.log(1e-3))   # softplus(dt_bias) in [1e-3, 1e-1]
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["D"] = 1 + 0.1 * randn(H, dtype=torch.float32)
        dt = _DT[case["state"]]
        if op == "ssm":
            s["init"] = randn(seqs, H, P, N, dtype=dt, scale=0.3) if case["init"] else None
        else:
            s["state"] = randn(case["S"], H, P, N, dtype=dt, scale=0.3)
    if op == "gated_norm":
        T, R, D = case["T"], case["R"], case["D"]
        s["x"] = randn(1, T, R, D, scale=0.5)
        s["gate"] = randn(1, T, R * D + case["extra"])[..., :R * D].unflatten(-1, (R, D))
        s["weight"] = 1 + randn(R, D, dtype=torch.float32, scale=0.1)
    if op == "residual_norm":
        T, D = case["T"], case["D"]
        s["x"], s["residual"] = randn(1, T, D), randn(1, T, D, dtype=_DT[case["residual"]], scale=2.0)
        s["weight"] = 1 + randn(D, dtype=torch.float32, scale=0.1)
        s["post"] = 1 + randn(D, dtype=torch.float32, scale=0.1) if case["post"] else None
        s["gate"] = randn(1, T, D) if case["gate"] else None
        s["chan"] = randn(D, dtype=torch.float32, scale=0.3) if case["chan"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "conv":
        s["out"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        s["final"] = torch.empty(case["varlen"] or case["B"], case["W"] - 1, case["C"], dtype=torch.bfloat16, device="cuda")
    elif op == "conv_step":
        s["out"] = torch.empty_like(s["x"])
    elif op in ("ssm", "ssm_step"):
        s["out"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        if op == "ssm":
            S = case["varlen"] or case["B"]
            s["final"] = torch.empty(S, case["H"], case["P"], N, dtype=_DT[case["state"]], device="cuda")
            s["workspace"] = None
    elif op == "gated_norm":
        s["out"] = torch.empty_like(s["x"])
    else:
        s["out"], s["residual_out"] = torch.empty_like(s["x"]), torch.empty_like(s["residual"])
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import gated_linear_attention_kda_gb300 as kda
    case = s["case"]
    op = case["op"]
    if op == "conv":
        kda.conv(s["x"], s["weight"], s["out"], s["bias"], silu=case["silu"], initial_state=s["init"],
                 final_state=s["final"], cu_seqlens=s["cu"])
        return {"out": s["out"], "state": s["final"]}
    if op == "conv_step":
        kda.conv_step(s["x"], s["weight"], s["out"], s["state"], s["bias"], silu=case["silu"])
        return {"out": s["out"], "state": s["state"]}
    if op == "ssm":
        if s["workspace"] is None:  # room for the states of a split time axis: a user's program keeps it between calls
            n = kda.ssm_workspace_bytes(case["varlen"] or case["B"], case["B"] * case["T"], case["H"], case["P"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        kda.ssm(s["x"], s["dt"], s["b"], s["c"], s["out"], s["A_log"], s["D"], s["dt_bias"], initial_state=s["init"],
                final_state=s["final"], cu_seqlens=s["cu"], workspace=s["workspace"])
        return {"out": s["out"], "state": s["final"]}
    if op == "ssm_step":
        kda.ssm_step(s["x"], s["dt"], s["b"], s["c"], s["out"], s["state"], s["A_log"], s["D"], s["dt_bias"])
        return {"out": s["out"], "state": s["state"]}
    if op == "gated_norm":
        kda.gated_norm(s["x"], s["gate"], s["weight"], s["out"], act=case["act"], gate_first=case["gate_first"], eps=EPS)
        return s["out"]
    kda.residual_norm(s["x"], s["residual"], s["residual_out"], s["weight"], s["out"], post_weight=s["post"],
                      gate=s["gate"], act=case["gate"] or "none", channel_scale=s["chan"], alpha=case["alpha"], eps=EPS)
    return {"out": s["out"], "residual": s["residual_out"]}


# ------------------------------------------------------------------------------------------ plain forms (32 bits)

def _pad_index(lengths, device):
    """[sequences, longest] positions of a packed token axis (clamped past an end) and which of them are tokens."""
    n = torch.tensor(lengths, device=device)
    t = torch.arange(max(lengths), device=device)
    live = t[None] < n[:, None]
    start = torch.cumsum(n, 0) - n
    return torch.where(live, start[:, None] + t[None], 0), live


def _conv_rows(ext, weight, bias, silu, W):
    """ext: [S, W - 1 + T, C] rows with the initial state in front."""
    T = ext.shape[1] - (W - 1)
    u = bias + sum(ext[:, k:k + T] * weight[:, k] for k in range(W))
    return u / (1 + torch.exp(-u)) if silu else u


def _plain_conv(s):
    case, W = s["case"], s["case"]["W"]
    x = s["x"].float()
    seqs = case["varlen"] or case["B"]
    init = s["init"].float() if s["init"] is not None else x.new_zeros(seqs, W - 1, case["C"])
    if s["lengths"] is None:
        ext = torch.cat([init, x], 1)
        return {"out": _conv_rows(ext, s["weight"], s["bias"], case["silu"], W).bfloat16(),
                "state": ext[:, ext.shape[1] - (W - 1):].bfloat16()}
    at, live = _pad_index(s["lengths"], x.device)
    ext = torch.cat([init, x[0][at]], 1)
    out = _conv_rows(ext, s["weight"], s["bias"], case["silu"], W)[live][None]
    last = torch.tensor(s["lengths"], device=x.device)[:, None] + torch.arange(W - 1, device=x.device)
    return {"out": out.bfloat16(), "state": torch.gather(ext, 1, last[..., None].expand(-1, -1, case["C"])).bfloat16()}


def _plain_conv_step(s):
    case = s["case"]
    ext = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    out = _conv_rows(ext, s["weight"], s["bias"], case["silu"], case["W"])[:, 0]
    s["state"].copy_(ext[:, 1:])  # the step's state is updated in place
    return {"out": out.bfloat16(), "state": s["state"]}


def _step_sizes(s, dt):
    """Delta and the log decay of every token and head."""
    u = dt.float() + s["dt_bias"]
    delta = torch.clamp(u, min=0) + torch.log1p(torch.exp(-torch.abs(u)))
    return delta, -torch.exp(s["A_log"]) * delta


def _joined(decay, state):
    """Inclusive scan over axis 1 of (decay, state) pairs by doubling: state[i] holds what chunks 0..i leave."""
    n, step = state.shape[1], 1
    while step < n:
        state = torch.cat([state[:, :step], state[:, step:] + decay[:, step:, :, None, None] * state[:, :-step]], 1)
        decay = torch.cat([decay[:, :step], decay[:, step:] * decay[:, :-step]], 1)
        step *= 2
    return state


def _plain_scan(s, x, delta, a, b, c, init):
    """x [S, T, H, P], delta and a [S, T, H], b and c [S, T, G, N], T a multiple of CHUNK; chunked, all in 32 bits but the
    running sums of the log decay (64)."""
    S, T, H, P = x.shape
    G, nc = b.shape[2], T // CHUNK
    hg = H // G
    x = x.view(S, nc, CHUNK, G, hg, P)
    b, c = (v.view(S, nc, CHUNK, G, N) for v in (b, c))
    xd = x * delta.view(S, nc, CHUNK, G, hg, 1)
    cum = torch.cumsum(a.double().view(S, nc, CHUNK, G, hg), 2)
    diff = cum.permute(0, 1, 3, 4, 2)
    diff = (diff[..., :, None] - diff[..., None, :]).float()                    # [S, nc, G, hg, i, j]
    low = torch.ones(CHUNK, CHUNK, device=x.device, dtype=torch.bool).tril()
    m = torch.exp(torch.where(low, diff, -math.inf))
    m *= torch.einsum("sqign,sqjgn->sqgij", c, b)[:, :, :, None]
    y = torch.einsum("sqghij,sqjghp->sqighp", m, xd)
    del m, diff
    tail = torch.exp((cum[:, :, -1:] - cum).float())
    local = torch.einsum("sqjghp,sqjgn->sqghpn", xd * tail[..., None], b).reshape(S, nc, H, P, N)
    whole = torch.exp(cum[:, :, -1].float()).reshape(S, nc, H)
    first = local[:, :1] + whole[:, :1, :, None, None] * init[:, None]
    after = _joined(whole, torch.cat([first, local[:, 1:]], 1))
    before = torch.cat([init[:, None], after[:, :-1]], 1).view(S, nc, G, hg, P, N)
    y += torch.exp(cum.float())[..., None] * torch.einsum("sqign,sqghpn->sqighp", c, before)
    return (y + s["D"].view(G, hg, 1) * x).reshape(S, T, H, P), after[:, -1]


def _plain_ssm(s):
    case = s["case"]
    delta, a = _step_sizes(s, s["dt"])
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    at = live = None
    if s["lengths"] is not None:
        at, live = _pad_index(s["lengths"], x.device)
        delta, a = (torch.where(live[..., None], v[0][at], 0) for v in (delta, a))
        x, b, c = (v[0][at] for v in (x, b, c))
    T = x.shape[1]
    pad = -T % CHUNK
    if pad:  # tokens with no step size leave the state as it is
        x, b, c = (torch.nn.functional.pad(v, (0, 0, 0, 0, 0, pad)) for v in (x, b, c))
        delta, a = (torch.nn.functional.pad(v, (0, 0, 0, pad)) for v in (delta, a))
    init = s["init"].float() if s["init"] is not None else x.new_zeros(x.shape[0], case["H"], case["P"], N)
    y, fin = _plain_scan(s, x, delta, a, b, c, init)
    y = y[:, :T]
    return {"out": (y[live][None] if live is not None else y).bfloat16(), "state": fin.to(_DT[case["state"]])}


def _plain_ssm_step(s):
    case = s["case"]
    delta, a = _step_sizes(s, s["dt"])
    hg = case["H"] // case["G"]
    b, c = (s[k].float().repeat_interleave(hg, 1) for k in ("b", "c"))
    x = s["x"].float()
    state = s["state"].float() * torch.exp(a)[..., None, None] + (delta[..., None] * x)[..., None] * b[:, :, None]
    out = (state * c[:, :, None]).sum(-1) + s["D"][:, None] * x
    s["state"].copy_(state)  # in place
    return {"out": out.bfloat16(), "state": s["state"]}


def _act(z, act):
    return z / (1 + torch.exp(-z)) if act == "silu" else 1 / (1 + torch.exp(-z)) if act == "sigmoid" else z


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_gated_norm(s):
    case = s["case"]
    x, z = s["x"].float(), _act(s["gate"].float(), case["act"])
    return ((_rms(x * z) * s["weight"]) if case["gate_first"] else (_rms(x) * s["weight"] * z)).bfloat16()


def _plain_residual_norm(s):
    case = s["case"]
    u = s["x"].float()
    if s["post"] is not None:
        u = _rms(u) * s["post"]
    if s["gate"] is not None:
        u = u * _act(s["gate"].float(), case["gate"])
    if s["chan"] is not None:
        u = u * s["chan"]
    r = s["residual"].float() + case["alpha"] * u
    return {"out": (_rms(r) * s["weight"]).bfloat16(), "residual": r.to(s["residual"].dtype)}


_PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "ssm": _plain_ssm, "ssm_step": _plain_ssm_step,
          "gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm}


# ------------------------------------------------------------------------------------------ definitions (64 bits)

def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    op = case["op"]
    sig = lambda z: torch.sigmoid(z)  # noqa: E731
    if op in ("conv", "conv_step"):
        W = case["W"]
        rows = [s["x"][i] for i in range(case["B"])] if op == "conv" else [r[None] for r in s["x"]]
        if op == "conv" and s["lengths"] is not None:
            rows = list(torch.split(s["x"][0], s["lengths"]))
        before = s["init"] if op == "conv" else s["state"]
        outs, states = [], []
        for i, r in enumerate(rows):
            e = torch.cat([before[i] if before is not None else r.new_zeros(W - 1, case["C"]), r])
            u = s["bias"].expand(r.shape).clone()
            for k in range(W):
                u += e[k:k + r.shape[0]] * s["weight"][:, k]
            outs.append(u * sig(u) if case["silu"] else u)
            states.append(e[-(W - 1):])
        out = torch.cat(outs) if op == "conv_step" else torch.cat(outs)[None] if s["lengths"] else torch.stack(outs)
        return {"out": out, "state": torch.stack(states)}
    if op in ("ssm", "ssm_step"):
        H, P, hg = case["H"], case["P"], case["H"] // case["G"]
        if op == "ssm_step":
            tok, state = {k: s[k][:, None] for k in ("x", "b", "c", "dt")}, s["state"]
            lengths = None
        else:
            lengths = s["lengths"]
            tok = {k: s[k] for k in ("x", "b", "c", "dt")}
            if lengths is not None:
                tok = {k: torch.nn.utils.rnn.pad_sequence(torch.split(v[0], lengths), batch_first=True) for k, v in tok.items()}
            state = s["init"] if s["init"] is not None else tok["x"].new_zeros(tok["x"].shape[0], H, P, N)
        S, T = tok["x"].shape[:2]
        delta = torch.logaddexp(tok["dt"] + s["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
        if lengths is not None:
            n = torch.tensor(lengths, device="cuda")
            delta = delta * (torch.arange(T, device="cuda") < n[:, None])[..., None]  # past an end nothing moves
        keep = torch.exp(-torch.exp(s["A_log"]) * delta)
        dx = delta[..., None] * tok["x"]
        y = torch.empty(S, T, H, P, dtype=torch.float64, device="cuda")
        state = state.clone()
        for t in range(T):
            bt, ct = (tok[k][:, t].repeat_interleave(hg, 1) for k in ("b", "c"))
            state *= keep[:, t, :, None, None]
            state.addcmul_(dx[:, t, :, :, None], bt[:, :, None])
            torch.matmul(state, ct[..., None], out=y[:, t, ..., None])
        y += s["D"][:, None] * tok["x"]
        if lengths is not None:
            y = torch.cat([y[i, :n] for i, n in enumerate(lengths)])[None]
        return {"out": y[:, 0] if op == "ssm_step" else y, "state": state}

    def normed(v):
        return v / torch.sqrt(torch.mean(v ** 2, -1, keepdim=True) + EPS)

    def gate(z, act):
        return z * sig(z) if act == "silu" else sig(z)

    if op == "gated_norm":
        z = gate(s["gate"], case["act"])
        return normed(s["x"] * z) * s["weight"] if case["gate_first"] else normed(s["x"]) * s["weight"] * z
    u = case["alpha"] * (normed(s["x"]) * s["post"] if s["post"] is not None else s["x"])
    u = u * gate(s["gate"], case["gate"]) if s["gate"] is not None else u
    r = s["residual"] + (u * s["chan"] if s["chan"] is not None else u)
    return {"out": normed(r) * s["weight"], "residual": r}


def work(case):
    op = case["op"]
    st = {"fp32": 4, "bf16": 2}
    if op == "conv":
        n, seqs = case["B"] * case["T"] * case["C"], case["varlen"] or case["B"]
        state = 2 * seqs * (case["W"] - 1) * case["C"]
        return {"bytes": 4 * n + state * (1 + case["states"]) + 4 * case["C"] * (case["W"] + 1), "flops": 2 * case["W"] * n}
    if op == "conv_step":
        n = case["S"] * case["C"]
        return {"bytes": 4 * n + 4 * n * (case["W"] - 1) + 4 * case["C"] * (case["W"] + 1), "flops": 2 * case["W"] * n}
    if op == "ssm":
        tok, seqs = case["B"] * case["T"], case["varlen"] or case["B"]
        state = seqs * case["H"] * case["P"] * N
        return {"bytes": tok * (4 * case["H"] * case["P"] + 4 * case["G"] * N + 2 * case["H"]) + state * st[case["state"]] * (1 + case["init"]),
                "flops": 4 * tok * case["H"] * case["P"] * N}
    if op == "ssm_step":
        state = case["S"] * case["H"] * case["P"] * N
        return {"bytes": 2 * state * st[case["state"]] + case["S"] * (4 * case["H"] * case["P"] + 4 * case["G"] * N + 2 * case["H"]),
                "flops": 4 * state}
    if op == "gated_norm":
        n = case["T"] * case["R"] * case["D"]
        return {"bytes": 6 * n + 4 * case["R"] * case["D"], "flops": 8 * n}
    n = case["T"] * case["D"]
    return {"bytes": n * (4 + 2 * st[case["residual"]] + 2 * bool(case["gate"])) + 4 * case["D"] * (1 + case["post"] + case["chan"]), "flops": 10 * n}
