"""Measured cases of the mixers that a hybrid stack puts beside KDA: the gated delta rule (``gdn``, ``gdn_step``), the
norm and rotation of queries and keys (``qk_rope``), appending to a paged cache (``kv_append``) and the attention of one
new token over it (``attn_step``). ``run`` computes a case with elementary torch operations (``own`` false) or with this
framework's calls (``own`` true); ``exact`` is the definition in 64 bits, token by token and row by row.

Sizes are the framework's own workloads (8 x 4096 tokens of 16 heads, 16 packed sequences of 32 heads, one
131072-token sequence of 32 heads, 128-sequence decode) with heads of 128 or 64 channels.
"""
import math

import torch

own = False

D = 128           # channels of a delta-rule head: keys and values
CHUNK = 64        # tokens per chunk of the plain delta rule
EPS = 1e-6


def listed():
    return [
        # a batch of prompts
        {"name": "gdn_b8_t4096_h16", "op": "gdn", "B": 8, "T": 4096, "H": 16, "HK": 16, "varlen": 0, "init": False,
         "state": "bf16", "l2": True},
        # packed prompts of ragged lengths, two value heads to a key head, states carried from an earlier call
        {"name": "gdn_varlen16_h32_hk16", "op": "gdn", "B": 1, "T": 65519, "H": 32, "HK": 16, "varlen": 16, "init": True,
         "state": "bf16", "l2": True},
        # one long document: few states, a long chain
        {"name": "gdn_b1_t131072_h32", "op": "gdn", "B": 1, "T": 131072, "H": 32, "HK": 32, "varlen": 0, "init": True,
         "state": "bf16", "l2": False},
        # a short prompt of one user, where latency counts
        {"name": "gdn_b1_t53_h8_hk4", "op": "gdn", "B": 1, "T": 53, "H": 8, "HK": 4, "varlen": 0, "init": True,
         "state": "bf16", "l2": True},
        # one decoding step of 128 sequences
        {"name": "gdn_step_s128_h16", "op": "gdn_step", "S": 128, "H": 16, "HK": 16, "state": "fp32", "l2": True},
        # queries and keys of a batch of prompts, slices of one projection, a quarter of each head turned
        {"name": "qk_rope_t32768_h16_hk4", "op": "qk_rope", "T": 32768, "H": 16, "HK": 4, "D": 128, "R": 32, "norm": True,
         "inter": False, "start": 0, "extra": 512},
        # the same for one decoding step, whole heads turned, far into long documents
        {"name": "qk_rope_s128_h32_hk8", "op": "qk_rope", "T": 128, "H": 32, "HK": 8, "D": 128, "R": 128, "norm": True,
         "inter": False, "start": 131072, "extra": 1024},
        # packed prompts behind what the cache holds of each sequence
        {"name": "kv_append_varlen16_hk8", "op": "kv_append", "T": 65519, "varlen": 16, "HK": 8, "D": 128, "R": 128,
         "norm": True, "inter": False, "start": 4096, "page": 64},
        # one decoding step of 128 sequences
        {"name": "kv_append_s128_hk4", "op": "kv_append", "T": 128, "varlen": 0, "HK": 4, "D": 128, "R": 64, "norm": True,
         "inter": False, "start": 4096, "page": 64},
        # one decoding step of 128 sequences of ragged lengths
        {"name": "attn_step_s128_h32_hk4", "op": "attn_step", "S": 128, "tokens": 524288, "H": 32, "HK": 4, "D": 128, "page": 64},
        # one step of one long document: few rows, a long axis
        {"name": "attn_step_s1_t131072_h32_hk8", "op": "attn_step", "S": 1, "tokens": 131072, "H": 32, "HK": 8, "D": 128,
         "page": 128},
        # a few short conversations, where latency counts
        {"name": "attn_step_s8_t4001_h16_hk2", "op": "attn_step", "S": 8, "tokens": 4001, "H": 16, "HK": 2, "D": 64, "page": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["gdn", "gdn", "gdn", "gdn_step", "qk_rope", "kv_append", "attn_step", "attn_step"])
    if op in ("gdn", "gdn_step"):
        per = rng.choice([1, 1, 2, 4])
        HK = _log_int(rng, 1, 32 // per)
        base = {"op": op, "H": per * HK, "HK": HK, "l2": rng.random() < 0.6}
        if op == "gdn_step":
            return {"S": _log_int(rng, 1, 128), "state": rng.choice(["fp32", "bf16"]), **base}
        varlen = rng.choice([0, 0, rng.randint(2, 24)])
        T = _log_int(rng, 1, min(131072, (1 << 21) // base["H"]))
        B = 1 if varlen else _log_int(rng, 1, max(1, min(16, (1 << 21) // (base["H"] * T))))
        return {"B": B, "T": max(T, varlen), "varlen": varlen, "init": rng.random() < 0.5, "state": "bf16", **base}
    HK = _log_int(rng, 1, 8)
    H, hd = HK * rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "attn_step":
        S = _log_int(rng, 1, 128)
        tokens = _log_int(rng, 4 * S, min(S * 16384, 131072) if S < 8 else min(S * 16384, (1 << 22) // HK // (hd // 64)))
        return {"op": op, "S": S, "tokens": tokens, "H": H, "HK": HK, "D": hd, "page": rng.choice([16, 32, 64, 128])}
    R, inter, norm = 16 * rng.randint(1, hd // 16), rng.random() < 0.3, rng.random() < 0.7
    if op == "qk_rope":
        return {"op": op, "T": _log_int(rng, 1, 32768), "H": H, "HK": HK, "D": hd, "R": R, "norm": norm, "inter": inter,
                "start": rng.choice([0, rng.randint(1, 1 << 20)]), "extra": rng.choice([0, 8 * rng.randint(1, 64)])}
    varlen = rng.choice([0, rng.randint(2, 24)])
    return {"op": op, "T": max(varlen, _log_int(rng, 1, 65536 if varlen else 256)), "varlen": varlen, "HK": HK, "D": hd, "R": R,
            "norm": norm, "inter": inter, "start": rng.choice([0, rng.randint(1, 4096)]), "page": rng.choice([16, 32, 64, 128])}


_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _lengths(n, T, seed):
    """``n`` positive lengths that add up to ``T``, spread as those of a batch of prompts are."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=gen).double() + 0.02
    ends = torch.floor(torch.cumsum(w, 0) / w.sum() * (T - n)).long() + torch.arange(1, n + 1)
    ends[-1] = T
    return [int(v) for v in torch.diff(ends, prepend=ends.new_zeros(1))]


def _pages(case, held, g):
    """A table of distinct pages in no order for sequences that hold ``held`` tokens, and how many pages there are: as
    many as these sequences need at most. Entries behind a sequence's last page are -1."""
    need = [(n + case["page"] - 1) // case["page"] for n in held]
    total = sum(held) // case["page"] + len(held)
    order = torch.randperm(total, generator=g, device="cuda")[:sum(need)].to(torch.int32)
    table = torch.full((len(held), max(need)), -1, dtype=torch.int32, device="cuda")
    live = torch.arange(max(need), device="cuda") < torch.tensor(need, device="cuda")[:, None]
    table[live] = order
    return table, total


def _inv_freq(R, base=500000.0):
    i = torch.arange(0, R, 2, dtype=torch.float64, device="cuda")
    return (base ** (-i / R)).float()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32).mul_(scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    op, s = case["op"], {}
    if op in ("gdn", "gdn_step"):
        H, HK = case["H"], case["HK"]
        tok = (case["B"], case["T"]) if op == "gdn" else (case["S"],)
        if op == "gdn":
            s["lengths"], s["cu"] = None, None
            if case["varlen"]:
                s["lengths"] = _lengths(case["varlen"], case["T"], seed)
                s["cu"] = torch.tensor([0] + s["lengths"], dtype=torch.int64).cumsum(0).cuda()
        # q, k and v are slices of one row of the convolution's output, as a layer has them
        qkv = randn(*tok, (2 * HK + H) * D)
        q, k, v = qkv.split([HK * D, HK * D, H * D], -1)
        if not case["l2"]:  # normalised ahead of the call
            for t in (q, k):
                u = t.unflatten(-1, (HK, D)).float()
                t.copy_((u * torch.rsqrt((u * u).sum(-1, keepdim=True) + EPS)).flatten(-2))
        s["q"], s["k"], s["v"] = q.unflatten(-1, (HK, D)), k.unflatten(-1, (HK, D)), v.unflatten(-1, (H, D))
        s["a"], s["beta"] = randn(*tok, H), randn(*tok, H)
        s["A_log"] = torch.log(1 + 15 * rand(H))
        step = torch.exp(rand(H) * math.log(100.0) + math.log(1e-3))   # softplus(dt_bias) in [1e-3, 1e-1]
        s["dt_bias"] = torch.log(torch.expm1(step))
        dt = _DT[case["state"]]
        if op == "gdn":
            s["init"] = randn(case["varlen"] or case["B"], H, D, D, dtype=dt, scale=0.1) if case["init"] else None
        else:
            s["state"] = randn(case["S"], H, D, D, dtype=dt, scale=0.1)
        return s
    if op == "attn_step":
        S, H, HK, hd = case["S"], case["H"], case["HK"], case["D"]
        s["lengths"] = _lengths(S, case["tokens"], seed)
        s["table"], total = _pages(case, s["lengths"], g)
        cache = randn(total, 2, HK, case["page"], hd)  # keys and values of a page side by side
        s["k_cache"], s["v_cache"] = cache[:, 0], cache[:, 1]
        s["q"] = randn(S, H, hd)
        s["positions"] = torch.tensor(s["lengths"], dtype=torch.int64, device="cuda") - 1
        return s
    T, HK, hd = case["T"], case["HK"], case["D"]
    s["inv_freq"] = _inv_freq(case["R"])
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (1 + randn(hd, dtype=torch.float32, scale=0.1) for _ in range(2))
    else:
        s["q_weight"] = s["k_weight"] = None
    if op == "qk_rope":
        H = case["H"]
        row = randn(1, T, (H + HK) * hd + case["extra"], scale=2.0)
        s["q"] = row[..., :H * hd].unflatten(-1, (H, hd))
        s["k"] = row[..., H * hd:(H + HK) * hd].unflatten(-1, (HK, hd))
        s["positions"] = case["start"] + torch.arange(T, device="cuda")[None]
        return s
    row = randn(T, 2 * HK * hd, scale=2.0)
    k, v = row.split(HK * hd, -1)
    s["k"], s["v"] = k.unflatten(-1, (HK, hd)), v.unflatten(-1, (HK, hd))
    lens = _lengths(case["varlen"], T, seed) if case["varlen"] else [1] * T
    before = torch.tensor(_lengths(len(lens), len(lens) * (1 + case["start"] // 2), seed + 1), device="cuda") - 1
    lens = torch.tensor(lens, device="cuda")
    s["seq"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
    cu = torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0)])
    s["positions"] = before[s["seq"]] + torch.arange(T, device="cuda") - cu[s["seq"]]
    s["table"], total = _pages(case, (before + lens).tolist(), g)
    cache = randn(total, 2, HK, case["page"], hd)
    s["k_cache"], s["v_cache"] = cache[:, 0], cache[:, 1]
    s["cu"] = cu if case["varlen"] else None
    if case["varlen"]:
        s["k"], s["v"], s["positions"] = s["k"][None], s["v"][None], s["positions"][None]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], op = case, case["op"]
    if op in ("gdn", "gdn_step"):
        s["out"] = torch.empty(s["v"].shape, dtype=torch.bfloat16, device="cuda")
        if op == "gdn":
            s["final"] = torch.empty(case["varlen"] or case["B"], case["H"], D, D, dtype=_DT[case["state"]], device="cuda")
    elif op == "qk_rope":
        s["q_out"], s["k_out"] = (torch.empty(s[n].shape, dtype=torch.bfloat16, device="cuda") for n in ("q", "k"))
    elif op == "attn_step":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["S"], case["H"], device="cuda")
        s["workspace"] = None
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import gated_linear_attention_kda_gb300 as kda
    case = s["case"]
    op = case["op"]
    if op == "gdn":
        kda.gdn(s["q"], s["k"], s["v"], s["a"], s["beta"], D ** -0.5, s["out"], s["A_log"], s["dt_bias"],
                initial_state=s["init"], final_state=s["final"], cu_seqlens=s["cu"], qk_l2norm=case["l2"])
        return {"out": s["out"], "state": s["final"]}
    if op == "gdn_step":
        kda.gdn_step(s["q"], s["k"], s["v"], s["a"], s["beta"], D ** -0.5, s["out"], s["state"], s["A_log"], s["dt_bias"],
                     qk_l2norm=case["l2"])
        return {"out": s["out"], "state": s["state"]}
    if op == "qk_rope":
        kda.qk_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                    norm=case["norm"], interleaved=case["inter"], eps=EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "kv_append":
        kda.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["positions"], s["inv_freq"], s["k_weight"],
                      norm=case["norm"], interleaved=case["inter"], eps=EPS, cu_seqlens=s["cu"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["workspace"] is None:  # room for the parts of a split cache: a user's program keeps it between calls
        n = kda.attn_step_workspace_bytes(case["S"], case["H"], case["HK"], case["D"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kda.attn_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["positions"], s["out"], case["D"] ** -0.5, lse=s["lse"],
                  workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------ plain forms (32 bits)

def _pad_index(lengths, device):
    """[sequences, longest] positions of a packed token axis (clamped past an end) and which of them are tokens."""
    n = torch.tensor(lengths, device=device)
    t = torch.arange(max(lengths), device=device)
    live = t[None] < n[:, None]
    start = torch.cumsum(n, 0) - n
    return torch.where(live, start[:, None] + t[None], 0), live


def _gate(s, a, beta):
    """The log decay and the step of every token and head."""
    u = a.float() + s["dt_bias"]
    delta = torch.clamp(u, min=0) + torch.log1p(torch.exp(-torch.abs(u)))
    return -torch.exp(s["A_log"]) * delta, 1 / (1 + torch.exp(-beta.float()))


def _heads(s, t):
    """Queries or keys in 32 bits, normalised where the call does it, one per value head."""
    t = t.float()
    if s["case"]["l2"]:
        t = t * torch.rsqrt((t * t).sum(-1, keepdim=True) + EPS)
    return t.repeat_interleave(s["case"]["H"] // s["case"]["HK"], -2)


def _plain_gdn(s):
    case = s["case"]
    q, k, v = _heads(s, s["q"]), _heads(s, s["k"]), s["v"].float()
    g, b = _gate(s, s["a"], s["beta"])
    live = None
    if s["lengths"] is not None:
        at, live = _pad_index(s["lengths"], v.device)
        q, k, v = (t[0][at] for t in (q, k, v))
        g, b = (torch.where(live[..., None], t[0][at], 0) for t in (g, b))
    S, T, H = v.shape[:3]
    pad = -T % CHUNK  # tokens with no step and no decay leave the state as it is
    if pad:
        q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad)) for t in (q, k, v))
        g, b = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (g, b))
    nc = (T + pad) // CHUNK
    q, k, v = (t.view(S, nc, CHUNK, H, D).transpose(2, 3) for t in (q, k, v))       # [S, nc, H, C, D]
    g, b = (t.view(S, nc, CHUNK, H).transpose(2, 3) for t in (g, b))                # [S, nc, H, C]
    cum = torch.cumsum(g.double(), -1)
    diff = (cum[..., :, None] - cum[..., None, :]).float()
    low = torch.ones(CHUNK, CHUNK, device=v.device, dtype=torch.bool).tril()
    m = torch.exp(torch.where(low, diff, -math.inf))
    del diff
    a = torch.matmul(k, k.transpose(-1, -2)) * m * b[..., None]
    t = torch.eye(CHUNK, device=v.device).expand(a.shape).contiguous()
    for i in range(1, CHUNK):  # (I + strictly lower a)^-1, row by row
        t[..., i, :i] = -torch.matmul(a[..., i:i + 1, :i], t[..., :i, :i])[..., 0, :]
    del a
    e = torch.exp(cum.float())[..., None]
    u = torch.matmul(t, v * b[..., None])
    w = torch.matmul(t, k * (b[..., None] * e))
    p = torch.matmul(q, k.transpose(-1, -2)) * m
    del t, m
    qe, kt = q * e, k * torch.exp((cum[..., -1:] - cum).float())[..., None]
    last = e[..., -1:, :]
    state = s["init"].float() if s["init"] is not None else v.new_zeros(S, H, D, D)
    out = torch.empty_like(v)
    for i in range(nc):
        n = u[:, i] - torch.matmul(w[:, i], state.transpose(-1, -2))
        out[:, i] = torch.matmul(qe[:, i], state.transpose(-1, -2)) + torch.matmul(p[:, i], n)
        state = last[:, i] * state + torch.matmul(n.transpose(-1, -2), kt[:, i])
    out = (D ** -0.5 * out).transpose(2, 3).reshape(S, nc * CHUNK, H, D)[:, :T]
    return {"out": (out[live][None] if live is not None else out).bfloat16(), "state": state.to(_DT[case["state"]])}


def _plain_gdn_step(s):
    q, k, v = _heads(s, s["q"]), _heads(s, s["k"]), s["v"].float()
    g, b = _gate(s, s["a"], s["beta"])
    state = s["state"].float() * torch.exp(g)[..., None, None]
    n = b[..., None] * (v - (state * k[:, :, None]).sum(-1))
    state = state + n[..., None] * k[:, :, None]
    out = D ** -0.5 * (state * q[:, :, None]).sum(-1)
    s["state"].copy_(state)  # in place
    return {"out": out.bfloat16(), "state": s["state"]}


def _turned(case, x, weight, positions, inv_freq):
    """Heads of x [..., heads, D] normed and turned, in 32 bits; the angles in 64."""
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    R = case["R"]
    angle = positions.double()[..., None, None] * inv_freq.double()
    c, d = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["inter"] else (x[..., :R // 2], x[..., R // 2:R])
    pair = (a * c - b * d, b * c + a * d)
    turned = torch.stack(pair, -1).flatten(-2) if case["inter"] else torch.cat(pair, -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_qk_rope(s):
    case = s["case"]
    return {n: _turned(case, s[n], s[n + "_weight"], s["positions"], s["inv_freq"]).bfloat16() for n in ("q", "k")}


def _plain_kv_append(s):
    case = s["case"]
    k = _turned(case, s["k"], s["k_weight"], s["positions"], s["inv_freq"]).bfloat16()
    pos = s["positions"].flatten()
    page, slot = s["table"][s["seq"], pos // case["page"]].long(), pos % case["page"]
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], s["v"])):
        cache[page, :, slot] = rows.reshape(-1, case["HK"], case["D"])  # in place
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn_step(s):
    case = s["case"]
    S, H, HK, hd = case["S"], case["H"], case["HK"], case["D"]
    table = s["table"].clamp(min=0).long()
    k, v = (s[n][table].transpose(2, 3).flatten(1, 2) for n in ("k_cache", "v_cache"))  # [S, tokens, HK, D]
    q = s["q"].float().view(S, HK, H // HK, hd)
    x = hd ** -0.5 * torch.einsum("shgd,sthd->shgt", q, k.float())
    x = torch.where(torch.arange(x.shape[-1], device=x.device) <= s["positions"][:, None, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("shgt,sthd->shgd", e / total, v.float())
    return {"out": out.reshape(S, H, hd).bfloat16(), "lse": (top + torch.log(total)).view(S, H)}


_PLAIN = {"gdn": _plain_gdn, "gdn_step": _plain_gdn_step, "qk_rope": _plain_qk_rope, "kv_append": _plain_kv_append,
          "attn_step": _plain_attn_step}


# ------------------------------------------------------------------------------------------ definitions (64 bits)

def _exact_rows(case, x, weight, positions, inv_freq):
    """One pair of channels at a time."""
    x = x.double()
    if case["norm"]:
        x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS) * weight.double()
    y, half = x.clone(), case["R"] // 2
    for i in range(half):
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        turn = torch.polar(torch.ones_like(positions, dtype=torch.float64), positions.double() * inv_freq[i].double())[..., None]
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "gdn" and case["T"] > 80000 and not case["varlen"]:
        return None  # token by token, half a minute
    s = _inputs(case, seed)
    if op in ("gdn", "gdn_step"):
        H, per = case["H"], case["H"] // case["HK"]
        f = {n: s[n].double() for n in ("q", "k", "v", "a", "beta")}
        if op == "gdn_step":
            f, lengths, state = {n: t[:, None] for n, t in f.items()}, None, s["state"].double()
        else:
            lengths = s["lengths"]
            if lengths is not None:
                f = {n: torch.nn.utils.rnn.pad_sequence(torch.split(t[0], lengths), batch_first=True) for n, t in f.items()}
            S = f["v"].shape[0]
            state = s["init"].double() if s["init"] is not None else f["v"].new_zeros(S, H, D, D)
        S, T = f["v"].shape[:2]
        keep = torch.exp(-torch.exp(s["A_log"].double()) * torch.logaddexp(f["a"] + s["dt_bias"].double(), f["a"].new_zeros(())))
        b = torch.sigmoid(f["beta"])
        if lengths is not None:  # past an end nothing moves
            live = (torch.arange(T, device="cuda") < torch.tensor(lengths, device="cuda")[:, None])[..., None]
            keep, b = torch.where(live, keep, 1.0), torch.where(live, b, 0.0)
        for n in ("q", "k") if case["l2"] else ():
            f[n] = f[n] / torch.sqrt((f[n] ** 2).sum(-1, keepdim=True) + EPS)
        out, state = torch.empty_like(f["v"]), state.clone()
        for t in range(T):
            kt, qt = (f[n][:, t].repeat_interleave(per, 1)[..., None] for n in ("k", "q"))
            state *= keep[:, t, :, None, None]
            miss = b[:, t, :, None, None] * (f["v"][:, t, :, :, None] - torch.matmul(state, kt))
            state.add_(torch.matmul(miss, kt.transpose(-1, -2)))
            out[:, t] = torch.matmul(state, qt)[..., 0] * D ** -0.5
        if lengths is not None:
            out = torch.cat([out[i, :n] for i, n in enumerate(lengths)])[None]
        return {"out": out[:, 0] if op == "gdn_step" else out, "state": state}
    if op == "qk_rope":
        return {n: _exact_rows(case, s[n], s[n + "_weight"], s["positions"], s["inv_freq"]) for n in ("q", "k")}
    if op == "kv_append":
        k = _exact_rows(case, s["k"], s["k_weight"], s["positions"], s["inv_freq"]).reshape(-1, case["HK"], case["D"])
        v = s["v"].double().reshape(k.shape)
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        pos, seq, table = s["positions"].flatten().tolist(), s["seq"].tolist(), s["table"].tolist()
        at = torch.tensor([table[i][p // case["page"]] * case["page"] + p % case["page"] for i, p in zip(seq, pos)], device="cuda")
        for cache, rows in ((k_cache, k), (v_cache, v)):
            for h in range(case["HK"]):
                flat = cache[:, h].reshape(-1, case["D"])
                flat[at] = rows[:, h]
                cache[:, h] = flat.view(cache[:, h].shape)
        return {"k_cache": k_cache, "v_cache": v_cache}
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    per = case["H"] // case["HK"]
    for i, n in enumerate(s["lengths"]):
        pages = s["table"][i, :(n + case["page"] - 1) // case["page"]].long()
        for h in range(case["HK"]):
            k, v = (s[c][pages, h].reshape(-1, case["D"])[:n].double() for c in ("k_cache", "v_cache"))
            x = s["q"][i, h * per:(h + 1) * per].double() @ k.T / math.sqrt(case["D"])
            lse[i, h * per:(h + 1) * per] = torch.logsumexp(x, -1)
            out[i, h * per:(h + 1) * per] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def work(case):
    op, st = case["op"], {"fp32": 4, "bf16": 2}
    if op in ("gdn", "gdn_step"):
        H, HK = case["H"], case["HK"]
        tok = case["B"] * case["T"] if op == "gdn" else case["S"]
        states = (case["varlen"] or case["B"]) * (1 + case["init"]) if op == "gdn" else 2 * case["S"]
        return {"bytes": tok * (4 * HK * D + 4 * H * D + 4 * H) + states * H * D * D * st[case["state"]],
                "flops": 6 * tok * H * D * D}
    if op == "qk_rope":
        n = case["T"] * (case["H"] + case["HK"]) * case["D"]
        return {"bytes": 4 * n + 8 * case["T"], "flops": 8 * n}
    if op == "kv_append":
        n = case["T"] * case["HK"] * case["D"]
        return {"bytes": 8 * n + 8 * case["T"] + 4 * case["T"] // case["page"], "flops": 8 * n}
    n = case["tokens"]
    return {"bytes": 4 * n * case["HK"] * case["D"] + 4 * n // case["page"] + 4 * case["S"] * case["H"] * case["D"] + 4 * case["S"] * case["H"],
            "flops": 4 * n * case["H"] * case["D"]}
