"""GPU tests of the operators around the mixer (convolution, state-space scan, gated norm, residual
norm) against plain 64-bit implementations (tests/block_ref.py).

Tolerances, fixed before the first run. A bf16 result is rounded once: 2^-8 of its value. Ahead of
that rounding:
* convolution and norms run in fp32 with hardware exponential and reciprocal: 2^-18 of the sum of
  the terms' magnitudes covers five fp32 roundings and the sigmoid's 2^-20;
* the scan's matrix form rounds the masked score matrix and the carried state to bf16 ahead of its
  products, 2^-8 of every term each: 2 * 2^-8 of the sum over absolute values. Independent roundings
  add as squares: three of rms 2^-8 / sqrt(3) give a relative L2 error of 2^-8;
* the scan's fp32 state: a decay over n tokens is exp2 of an fp32 sum of n <= 128 terms (its error
  n 2^-24 |E| 2^-|E| ln 2 <= 2^-18), and the increments are sums of exact products of bf16 parts;
  2^-16 of the sum over absolute values covers both with the roundings of the carried state."""
import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
NAN = float("nan")


@pytest.fixture(scope="module")
def kda():
    import gated_linear_attention_kda_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def wide(t, before, after):
    """The same values as a slice of a wider row whose other elements are NaN."""
    w = torch.full(t.shape[:-1] + (before + t.shape[-1] + after,), NAN, dtype=t.dtype, device=t.device)
    w[..., before:before + t.shape[-1]] = t
    return w[..., before:before + t.shape[-1]]


def close(got, ref, slack, what):
    err = (got.double() - ref).abs()
    ok = (err <= slack) & torch.isfinite(got.double())
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst {float((err - slack).nan_to_num(9e9).max()):.3e} over"


def cu_of(lengths):
    return torch.tensor([0] + list(lengths), dtype=torch.int64).cumsum(0).cuda()


# ------------------------------------------------------------------------------------- convolution

def check_conv(kda, B, T, C, W, silu=True, bias=True, init=True, lengths=None, strided=False, in_place=False, seed=0):
    g = gen(seed)
    x = randn(g, B, T, C)
    if strided:
        x = wide(x, 8, 24)
    w, bs = randn(g, C, W, dtype=torch.float32), randn(g, C, dtype=torch.float32) if bias else None
    cu = cu_of(lengths) if lengths is not None else None
    S = len(lengths) if lengths is not None else B
    st = randn(g, S, W - 1, C) if init else None
    ref, fin, mag = R.conv(x, w, bs, silu, st, cu)
    out = torch.full((B, T, C + (16 if strided else 0)), NAN, dtype=torch.bfloat16, device="cuda")[..., :C]
    final = st if in_place and init else torch.full((S, W - 1, C), NAN, dtype=torch.bfloat16, device="cuda")
    kda.conv(x, w, out, bs, silu=silu, initial_state=st, final_state=final, cu_seqlens=cu)
    kda.check_device_status()
    close(out, ref, HALF * ref.abs() + 2.0 ** -18 * mag + 1e-37, "out")
    assert torch.equal(final.double(), fin)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T,C", [(1, 8), (2, 40), (3, 64), (31, 2048), (33, 1032), (97, 8), (300, 4352)])
def test_conv(kda, W, T, C):
    check_conv(kda, 2, T, C, W, silu=(T % 2 == 1), bias=(C != 64), init=(T != 31), strided=(C == 1032), seed=T + C + W)


@pytest.mark.parametrize("lengths", [[1, 2, 0, 5, 31, 1, 1, 64], [0, 0, 7], [129, 0], [3]])
@pytest.mark.parametrize("in_place", [False, True])
def test_conv_varlen(kda, lengths, in_place):
    check_conv(kda, 1, sum(lengths), 72, 4, lengths=lengths, in_place=in_place, seed=len(lengths))


def test_conv_in_place_state_of_short_rows(kda):
    for T in (1, 2, 3):
        check_conv(kda, 5, T, 16, 4, in_place=True, seed=T)


def test_conv_does_not_mix_sequences_that_hold_nan(kda):
    """A sequence of NaN beside a sequence of numbers leaves the numbers' outputs and state alone."""
    g = gen(3)
    x = randn(g, 1, 40, 16)
    x[:, 17:29] = NAN
    w = randn(g, 16, 4, dtype=torch.float32)
    cu = cu_of([17, 12, 11])
    out, fin = torch.empty_like(x), torch.empty(3, 3, 16, dtype=torch.bfloat16, device="cuda")
    kda.conv(x, w, out, final_state=fin, cu_seqlens=cu)
    kda.check_device_status()
    assert torch.isfinite(out[:, :17]).all() and torch.isfinite(out[:, 29:]).all() and torch.isfinite(fin[[0, 2]]).all()
    assert torch.isnan(out[:, 17:29]).all()


def test_conv_empty_call(kda):
    x = torch.empty(2, 0, 24, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(24, 3, device="cuda")
    st = randn(gen(1), 2, 2, 24)
    fin = torch.full_like(st, NAN)
    kda.conv(x, w, torch.empty_like(x), initial_state=st, final_state=fin)
    assert torch.equal(fin, st)
    kda.conv(x, w, torch.empty_like(x), final_state=fin)
    assert not fin.any()


def test_conv_silu_tails(kda):
    """Large magnitudes of both signs: the tails of u sigmoid(u)."""
    x = torch.tensor([-3e38, -1e4, -90.0, -88.0, -60.0, -20.0, -1e-3, 0.0, 1e-3, 20.0, 90.0, 3e38], device="cuda").bfloat16()
    x = x.repeat_interleave(2)[None, None].contiguous()
    w = torch.zeros(24, 2, device="cuda")
    w[:, 1] = 1.0
    out = torch.empty_like(x)
    kda.conv(x, w, out)
    ref = x.double() * torch.sigmoid(x.double())
    close(out, ref, HALF * ref.abs() + 2e-36, "out")


@pytest.mark.parametrize("S,C,W", [(1, 8, 4), (3, 2048, 4), (130, 72, 2), (7, 264, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_conv_step(kda, S, C, W, in_place):
    """Steps that continue one another equal one prompt."""
    g = gen(S + C)
    x, w, b, st = randn(g, S, 5, C), randn(g, C, W, dtype=torch.float32), randn(g, C, dtype=torch.float32), randn(g, S, W - 1, C)
    ref, fin, mag = R.conv(x, w, b, True, st)
    state = st.clone()
    for t in range(5):
        xt = wide(x[:, t], 8, 8)
        out = xt if in_place else torch.full((S, C), NAN, dtype=torch.bfloat16, device="cuda")
        kda.conv_step(xt, w, out, state, b)
        close(out, ref[:, t], HALF * ref[:, t].abs() + 2.0 ** -18 * mag[:, t] + 1e-37, f"token {t}")
    assert torch.equal(state.double(), fin)


def test_conv_bad_bounds_are_flagged(kda):
    x = randn(gen(0), 1, 20, 8)
    w = torch.ones(8, 4, device="cuda")
    for bad in ([0, 25], [1, 20], [0, 12, 8, 20], [-3, 20], [0, 19]):
        out = torch.empty_like(x)
        fin = torch.zeros(len(bad) - 1, 3, 8, dtype=torch.bfloat16, device="cuda")
        kda.conv(x, w, out, final_state=fin, cu_seqlens=torch.tensor(bad, device="cuda"))
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_device_status()


# ------------------------------------------------------------------------------------------- scan

def ssm_inputs(g, B, T, H, P, G, strided=False, dt_scale=1.0):
    xbc = randn(g, B, T, H * P + 2 * G * 128)
    if strided:
        xbc = wide(xbc, 16, 8)
    x = xbc[..., :H * P].unflatten(-1, (H, P))
    b = xbc[..., H * P:H * P + G * 128].unflatten(-1, (G, 128))
    c = xbc[..., H * P + G * 128:].unflatten(-1, (G, 128))
    dt = randn(g, B, T, H, scale=dt_scale)
    if strided:
        dt = wide(dt, 1, 2)
    A_log = torch.log(1 + 15 * torch.rand(H, generator=g, device="cuda"))
    dt_bias = torch.rand(H, generator=g, device="cuda") * 4.6 - 6.9
    return x, dt, b, c, A_log, randn(g, H, dtype=torch.float32), dt_bias


_SDT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def check_states(got, fin, fmag, name):
    slack = 2.0 ** -16 * fmag + 1e-30
    if got.dtype == torch.bfloat16:
        slack = slack * (1 + HALF) + HALF * fin.abs()
    close(got, fin, slack, name)


def check_ssm(kda, B, T, H, P, G, state="fp32", init=True, lengths=None, strided=False, in_place=False, use_D=True,
              use_bias=True, workspace=True, seed=0, dt_scale=1.0):
    g = gen(seed)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, B, T, H, P, G, strided, dt_scale)
    D, dt_bias = D if use_D else None, dt_bias if use_bias else None
    cu = cu_of(lengths) if lengths is not None else None
    S = len(lengths) if lengths is not None else B
    st = randn(g, S, H, P, 128, dtype=_SDT[state], scale=0.3) if init else None
    ref, fin, mag, fmag = R.ssm(x, dt, b, c, A_log, D, dt_bias, st, cu)
    out = torch.full((B, T, H * P + (8 if strided else 0)), NAN, dtype=torch.bfloat16, device="cuda")[..., :H * P].unflatten(-1, (H, P))
    final = st if in_place and init else torch.full((S, H, P, 128), NAN, dtype=_SDT[state], device="cuda")
    ws = torch.full((kda.ssm_workspace_bytes(S, B * T, H, P),), 0xff, dtype=torch.uint8, device="cuda") if workspace else None
    kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, initial_state=st, final_state=final, cu_seqlens=cu, workspace=ws)
    kda.check_device_status()
    if T:
        close(out, ref, HALF * ref.abs() + 2 * HALF * (1 + HALF) * mag + 1e-30, "out")
        rel = float((out.double() - ref).norm() / ref.norm().clamp_min(1e-30))
        assert rel <= HALF, rel
    check_states(final, fin, fmag, "state")


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 127, 128, 129, 255, 300, 513])
def test_ssm_lengths(kda, T, P):
    check_ssm(kda, 2, T, 3, P, 1, seed=T + P, init=(T % 2 == 1), state="bf16" if T in (17, 300) else "fp32")


@pytest.mark.parametrize("H,G", [(1, 1), (4, 2), (6, 6), (8, 1)])
def test_ssm_groups(kda, H, G):
    check_ssm(kda, 1, 200, H, 64, G, seed=H + G, strided=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lengths", [[1, 2, 0, 130, 128, 1, 257], [0, 0, 5], [384, 0], [700]])
@pytest.mark.parametrize("P", [64, 128])
def test_ssm_varlen(kda, lengths, in_place, P):
    check_ssm(kda, 1, sum(lengths), 2, P, 1, lengths=lengths, in_place=in_place, seed=len(lengths) + P)


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("T,state", [(1500, "fp32"), (4000, "bf16")])
def test_ssm_long_chain_of_few_states(kda, T, state, workspace):
    check_ssm(kda, 1, T, 2, 128, 1, state=state, workspace=workspace, seed=T)


def test_ssm_many_states(kda):
    check_ssm(kda, 5, 140, 40, 64, 4, seed=9, use_D=False)


def test_ssm_optional_parameters(kda):
    check_ssm(kda, 1, 150, 2, 128, 1, use_D=False, use_bias=False, init=False, seed=4)


def test_ssm_strong_and_weak_decay(kda):
    """Step sizes from next to nothing (softplus of -20) to dozens, whose decay underflows."""
    check_ssm(kda, 1, 400, 4, 64, 1, dt_scale=20.0, use_bias=False, seed=11)


def test_ssm_continues_a_call_in_pieces(kda):
    """300 tokens in one call equal calls of 170, 1 and 129 tokens that hand the state on."""
    g = gen(5)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 2, 300, 3, 64, 1)
    ref, fin, mag, fmag = R.ssm(x, dt, b, c, A_log, D, dt_bias, None)
    state = torch.zeros(2, 3, 64, 128, device="cuda")
    for s0, s1 in ((0, 170), (170, 171), (171, 300)):
        cut = [v[:, s0:s1].contiguous() for v in (x, dt, b, c)]
        out = torch.empty_like(cut[0])
        kda.ssm(*cut, out, A_log, D, dt_bias, initial_state=state, final_state=state)
        kda.check_device_status()
        close(out, ref[:, s0:s1], HALF * ref[:, s0:s1].abs() + 2 * HALF * (1 + HALF) * mag[:, s0:s1], f"{s0}")
    check_states(state, fin, fmag, "state")


def test_ssm_does_not_mix_sequences_that_hold_nan_or_infinity(kda):
    g = gen(6)
    lengths = [70, 60, 150]
    x, dt, b, c, A_log, D, dt_bias = (v.clone() for v in ssm_inputs(g, 1, sum(lengths), 2, 64, 1))
    for v, bad in ((x, NAN), (dt, NAN), (b, float("inf")), (c, NAN)):
        v[:, 70:130] = bad
    out = torch.empty_like(x)
    fin = torch.empty(3, 2, 64, 128, device="cuda")
    kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, cu_seqlens=cu_of(lengths))
    kda.check_device_status()
    assert torch.isfinite(out[:, :70]).all() and torch.isfinite(out[:, 130:]).all() and torch.isfinite(fin[[0, 2]]).all()
    # NaN at one token reaches every later output of its sequence
    assert torch.isnan(out[:, 70:130]).all()


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("P,T,at", [(64, 300, 200), (128, 400, 130), (64, 5, 3), (128, 128, 127), (64, 1400, 700)])
@pytest.mark.parametrize("workspace", [False, True])
def test_ssm_a_non_finite_x_stays_in_its_channel_and_chunk(kda, P, T, at, bad, workspace):
    """NaN or infinity in one channel of x at one token: other channels and earlier chunks of 128 tokens (earlier tokens,
    where the call has no chunks) are as without it, and that channel's later outputs and its state hold no number."""
    g = gen(40 + T)
    x, dt, b, c, A_log, D, dt_bias = (v.clone() for v in ssm_inputs(g, 1, T, 2, P, 1))
    A_log -= 6  # weak decay: what was spoilt stays
    ws = torch.empty(max(16, kda.ssm_workspace_bytes(1, T, 2, P)), dtype=torch.uint8, device="cuda") if workspace else None

    def run():
        out, fin = torch.full_like(x, 7.0), torch.full((1, 2, P, 128), 7.0, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, workspace=ws)
        kda.check_device_status()
        return out, fin

    ref_out, ref_fin = run()
    x[0, at, 1, 9] = bad
    out, fin = run()
    same = torch.ones(1, T, 2, P, dtype=torch.bool, device="cuda")
    same[:, at // 128 * 128 if T > 8 else at:, 1, 9] = False
    assert torch.equal(out[same], ref_out[same])
    assert not torch.isfinite(out[0, at:, 1, 9]).any()
    rest = torch.ones(1, 2, P, dtype=torch.bool, device="cuda")
    rest[0, 1, 9] = False
    assert torch.equal(fin[rest], ref_fin[rest]) and not torch.isfinite(fin[0, 1, 9]).any()


@pytest.mark.parametrize("which", ["dt", "b", "c"])
@pytest.mark.parametrize("T,at", [(300, 200), (140, 131), (400, 40)])
def test_ssm_a_nan_never_reaches_earlier_tokens(kda, which, T, at):
    g = gen(60 + T)
    args = dict(zip(("x", "dt", "b", "c", "A_log", "D", "dt_bias"), (v.clone() for v in ssm_inputs(g, 1, T, 2, 64, 1))))
    out, ref = torch.empty_like(args["x"]), torch.empty_like(args["x"])
    kda.ssm(out=ref, **args)
    args[which][:, at] = NAN
    kda.ssm(out=out, **args)
    kda.check_device_status()
    assert torch.equal(out[:, :at], ref[:, :at]) and torch.isnan(out[:, at]).all()
    if which == "c":
        assert torch.equal(out[:, at + 1:], ref[:, at + 1:])
    else:
        assert torch.isnan(out[:, at:]).all()


def test_ssm_empty_call(kda):
    z = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    st = randn(gen(1), 2, 3, 64, 128, dtype=torch.float32)
    fin = torch.full_like(st, NAN)
    A = torch.zeros(3, device="cuda")
    args = (z(2, 0, 3, 64), z(2, 0, 3), z(2, 0, 1, 128), z(2, 0, 1, 128), z(2, 0, 3, 64), A)
    kda.ssm(*args, initial_state=st, final_state=fin)
    assert torch.equal(fin, st)
    kda.ssm(*args, final_state=fin)
    assert not fin.any()


def test_ssm_bad_bounds_are_flagged(kda):
    g = gen(7)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, 300, 2, 64, 1)
    for bad in ([0, 310], [1, 300], [0, 200, 150, 300], [-3, 300], [0, 299]):
        out = torch.empty(1, 300, 2, 64, dtype=torch.bfloat16, device="cuda")
        fin = torch.zeros(len(bad) - 1, 2, 64, 128, device="cuda")
        ws = torch.empty(kda.ssm_workspace_bytes(len(bad) - 1, 300, 2, 64), dtype=torch.uint8, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, cu_seqlens=torch.tensor(bad, device="cuda"), workspace=ws)
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_device_status()


@pytest.mark.parametrize("S,H,P,G,state", [(1, 1, 64, 1, "fp32"), (3, 4, 128, 2, "bf16"), (37, 6, 64, 3, "fp32"), (128, 2, 128, 1, "fp32")])
def test_ssm_step(kda, S, H, P, G, state):
    """Three steps against the recurrence; the step's own arithmetic is fp32 throughout."""
    g = gen(S + H)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, S, 3, H, P, G, strided=True)
    st = randn(g, S, H, P, 128, dtype=_SDT[state], scale=0.3)
    got = st.clone()
    for t in range(3):
        ref, fin, mag, fmag = R.ssm(*(v[:, t:t + 1] for v in (x, dt, b, c)), A_log, D, dt_bias, got)
        out = torch.full((S, H, P), NAN, dtype=torch.bfloat16, device="cuda")
        kda.ssm_step(x[:, t], dt[:, t], b[:, t], c[:, t], out, got, A_log, D, dt_bias)
        close(out, ref[:, 0], HALF * ref[:, 0].abs() + 2.0 ** -16 * mag[:, 0] + 1e-30, f"token {t}")
        check_states(got, fin, fmag, f"state {t}")


# ------------------------------------------------------------------------------------------ norms

@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("M,Rr,D", [(1, 1, 8), (5, 3, 24), (33, 16, 128), (7, 2, 264), (3, 1, 1000), (2, 2, 1032), (4, 1, 2048),
                                    (2, 1, 8192), (3, 1, 8200), (1, 1, 16384)])
def test_gated_norm(kda, M, Rr, D, act, gate_first):
    g = gen(M + D)
    x, z = randn(g, 1, M, Rr, D), wide(randn(g, 1, M, Rr * D), 8, 16).unflatten(-1, (Rr, D))
    w = 1 + randn(g, Rr, D, dtype=torch.float32, scale=0.2)
    if M % 2:
        w = w[0].contiguous()
    out = torch.full_like(x, NAN)
    kda.gated_norm(x, z, w, out, act=act, gate_first=gate_first)
    ref = R.gated_norm(x, z, w, act, gate_first, 1e-5)
    close(out, ref, (HALF + 2.0 ** -18) * ref.abs() + 1e-30, "out")


def test_gated_norm_in_place_and_zero_rows(kda):
    g = gen(2)
    x, z = randn(g, 6, 4, 128), randn(g, 6, 4, 128)
    x[2] = 0
    x[4, 1] = 0
    ref = R.gated_norm(x, z, None, "silu", False, 1e-6)
    for target in (x.clone(), z.clone()):
        a, b = (target, z) if torch.equal(target, x) else (x, target)
        kda.gated_norm(a, b, None, target, act="silu", eps=1e-6)
        close(target, ref, (HALF + 2.0 ** -18) * ref.abs() + 1e-30, "out")


def test_gated_norm_keeps_a_row_of_nan_to_itself(kda):
    g = gen(8)
    x, z = randn(g, 1, 9, 4, 128), randn(g, 1, 9, 4, 128)
    x[0, 3, 1, 5] = NAN
    out = torch.empty_like(x)
    kda.gated_norm(x, z, None, out)
    bad = torch.isnan(out).any(-1)
    assert int(bad.sum()) == 1 and bool(bad[0, 3, 1]) and torch.isnan(out[0, 3, 1]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,act,chan,alpha", [(False, None, False, 1.0), (True, None, False, 0.5), (True, "sigmoid", True, -0.25),
                                                 (False, "silu", True, 2.0), (True, "none", False, 1.0)])
@pytest.mark.parametrize("M,D", [(1, 8), (9, 136), (300, 1000), (5, 2048), (700, 2056), (3, 8192), (2, 16384)])
def test_residual_norm(kda, M, D, post, act, chan, alpha, dtype):
    g = gen(M + D)
    x, r = wide(randn(g, 1, M, D), 8, 0), wide(randn(g, 1, M, D, dtype=dtype, scale=2.0), 8, 8)
    w = 1 + randn(g, D, dtype=torch.float32, scale=0.2)
    pw = 1 + randn(g, D, dtype=torch.float32, scale=0.2) if post else None
    z = randn(g, 1, M, D) if act else None
    ch = randn(g, D, dtype=torch.float32) if chan else None
    ref, rr, mag = R.residual_norm(x, r, w, pw, z, act, ch, alpha, 1e-5)
    ro, out = torch.full((1, M, D), NAN, dtype=dtype, device="cuda"), torch.full((1, M, D), NAN, dtype=torch.bfloat16, device="cuda")
    kda.residual_norm(x, r, ro, w, out, post_weight=pw, gate=z, act=act or "none", channel_scale=ch, alpha=alpha)
    rslack = 2.0 ** -18 * mag + 1e-30
    close(ro, rr, rslack + (HALF * rr.abs() if dtype == torch.bfloat16 else 0), "residual")
    # the sum's own rounding error, carried through the norm of its row, comes on top
    inv = 1 / torch.sqrt((rr * rr).mean(-1, keepdim=True) + 1e-5)
    close(out, ref, (HALF + 2.0 ** -18) * ref.abs() + 2 * rslack * inv * w.double().abs(), "out")


def test_residual_norm_in_place_and_single_outputs(kda):
    g = gen(12)
    x, r = randn(g, 4, 512), randn(g, 4, 512, dtype=torch.float32)
    w = torch.ones(512, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(r)
    kda.residual_norm(x, r, b, w, a)
    r2, x2 = r.clone(), x.clone()
    kda.residual_norm(x2, r2, r2, w, x2)  # residual in place, out over x
    assert torch.equal(r2, b) and torch.equal(x2, a)
    only = torch.empty_like(r)
    kda.residual_norm(x, r, only)
    assert torch.equal(only, b)
    last = torch.empty_like(x)
    kda.residual_norm(x, r, None, w, last)
    assert torch.equal(last, a)


def test_residual_norm_cancelling_rows(kda):
    """x = -residual leaves a row of zeros and a norm of zeros."""
    x = randn(gen(13), 3, 256)
    r = -x.float()
    ro, out = torch.full_like(r, NAN), torch.full_like(x, NAN)
    kda.residual_norm(x, r, ro, None, out)
    assert not ro.any() and not out.any()


# ---------------------------------------------------------------------------- streams and graphs

def _calls(kda, g):
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, 200, 2, 64, 1)
    cw, cb, cst = randn(g, 128, 4, dtype=torch.float32), None, randn(g, 1, 3, 128)
    flat = x.reshape(1, 200, 128).contiguous()
    o = {"conv": torch.empty_like(flat), "cfin": torch.empty_like(cst), "ssm": torch.empty(1, 200, 2, 64, dtype=torch.bfloat16, device="cuda"),
         "sfin": torch.empty(1, 2, 64, 128, device="cuda"), "norm": torch.empty(1, 200, 2, 64, dtype=torch.bfloat16, device="cuda"),
         "res": torch.empty_like(flat), "pre": torch.empty_like(flat)}
    ws = torch.empty(max(1, kda.ssm_workspace_bytes(1, 200, 2, 64)), dtype=torch.uint8, device="cuda")
    w = torch.ones(128, device="cuda")

    def run():
        kda.conv(flat, cw, o["conv"], cb, initial_state=cst, final_state=o["cfin"])
        kda.ssm(o["conv"].unflatten(-1, (2, 64)), dt, b, c, o["ssm"], A_log, D, dt_bias, final_state=o["sfin"], workspace=ws)
        kda.gated_norm(o["ssm"], x, None, o["norm"], act="silu")
        kda.residual_norm(o["norm"].flatten(2), flat, o["res"], w, o["pre"])
    return run, o


def test_calls_replay_from_a_cuda_graph(kda):
    run, o = _calls(kda, gen(20))
    run()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in o.items()}
    for v in o.values():
        v.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    kda.check_device_status()
    for k in ref:
        assert torch.equal(o[k], ref[k]), k


def test_calls_run_on_the_current_stream(kda):
    run, o = _calls(kda, gen(21))
    run()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in o.items()}
    for v in o.values():
        v.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    for k in ref:
        assert torch.equal(o[k], ref[k]), k


def test_repeated_calls_are_bitwise_equal(kda):
    g = gen(22)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, 1000, 3, 128, 1)
    ws = torch.empty(max(1, kda.ssm_workspace_bytes(1, 1000, 3, 128)), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(3):
        out, fin = torch.empty(1, 1000, 3, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 3, 128, 128, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, workspace=ws)
        got.append((out, fin))
    kda.check_device_status()
    for o, f in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(f, got[0][1])


# ------------------------------------------------------------------- refusals on tensors, far offsets

def test_calls_refuse_mismatched_tensors(kda):
    g = gen(30)
    x = randn(g, 2, 6, 64)
    w = randn(g, 64, 4, dtype=torch.float32)
    out = torch.full_like(x, NAN)
    for bad, match in ((dict(weight=w.bfloat16()), "weight must be torch.float32"), (dict(weight=w[:, :1].contiguous()), "W must be 2, 3 or 4"),
                       (dict(out=out.float()), "out must be torch.bfloat16"), (dict(out=out[:, :3]), "out has shape"),
                       (dict(initial_state=torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda")), "initial_state has shape"),
                       (dict(x=x.expand(2, 6, 64)[:, :, :60], out=out[:, :, :60], weight=w[:60].contiguous()), "multiple of 8"),
                       (dict(out=x), "must not share memory"), (dict(bias=torch.zeros(64)), "bias must be a CUDA tensor"),
                       (dict(cu_seqlens=torch.tensor([0, 12], device="cuda")), "varlen mode needs B == 1")):
        args = {**dict(x=x, weight=w, out=out), **bad}
        with pytest.raises(ValueError, match=match):
            kda.conv(**args)
    assert torch.isnan(out).all()
    xs, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, 300, 4, 64, 2)
    o = torch.empty(1, 300, 4, 64, dtype=torch.bfloat16, device="cuda")
    need = kda.ssm_workspace_bytes(1, 300, 4, 64)
    for bad, match in ((dict(A_log=None), "A_log is required"), (dict(c=c[..., :1, :]), "c has shape"), (dict(D=D[:3].contiguous()), "D has shape"),
                       (dict(x=xs[:, ::2], dt=dt[:, ::2], b=b[:, ::2], c=c[:, ::2], out=xs[:, 1::2]), "token strides|share memory|out must"),
                       (dict(final_state=torch.empty(1, 4, 64, 128, dtype=torch.float16, device="cuda")), "final_state must be")):
        args = {**dict(x=xs, dt=dt, b=b, c=c, out=o, A_log=A_log), **bad}
        if "x" in bad:  # every other token, written to the tokens between: rows that interleave are allowed
            kda.ssm(**args)
            continue
        with pytest.raises(ValueError, match=match):
            kda.ssm(**args)
    if need:
        with pytest.raises(ValueError, match="workspace of"):
            kda.ssm(xs, dt, b, c, o, A_log, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    kda.check_device_status()


def test_conv_offsets_past_32_bits(kda):
    """Token strides that put the last rows more than 2^32 elements from the first."""
    T, C, stride = 70000, 16, 65536
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, T, C), (T * stride, stride, 1))
    g = gen(31)
    x.copy_(randn(g, 1, T, C))
    w = randn(g, C, 4, dtype=torch.float32)
    ref, fin, mag = R.conv(x, w, None, True, None)
    out = x.as_strided((1, T, C), (T * stride, stride, 1), 64)  # 64 channels further on in the same rows
    final = torch.empty(1, 3, C, dtype=torch.bfloat16, device="cuda")
    kda.conv(x, w, out, final_state=final)
    close(out, ref, HALF * ref.abs() + 2.0 ** -18 * mag + 1e-37, "out")
    assert torch.equal(final.double(), fin)


def test_ssm_offsets_past_32_bits(kda):
    T, stride = 70000, 65536
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    view = lambda off, *s: big.as_strided((1, T, *s), (T * stride, stride) + ((s[1], 1) if len(s) == 2 else (1,)), off)  # noqa: E731
    g = gen(32)
    x, b, c, dt, out = view(0, 1, 64), view(64, 1, 128), view(192, 1, 128), view(321, 1), view(512, 1, 64)
    for v in (x, b, c):
        v.copy_(randn(g, *v.shape))
    dt.copy_(randn(g, 1, T, 1))
    A_log = torch.zeros(1, device="cuda")
    tail = slice(T - 300, T)
    # the decay over a few thousand tokens leaves nothing of what came before: the tail's own recurrence is the reference
    near = [v[:, T - 6000:].contiguous() for v in (x, dt, b, c)]
    ref, fin, mag, fmag = R.ssm(*near, A_log, None, None, None)
    ws = torch.empty(max(16, kda.ssm_workspace_bytes(1, T, 1, 64)), dtype=torch.uint8, device="cuda")
    final = torch.empty(1, 1, 64, 128, device="cuda")
    kda.ssm(x, dt, b, c, out, A_log, final_state=final, workspace=ws)
    kda.check_device_status()
    r, m = ref[:, -300:], mag[:, -300:]
    close(out[:, tail], r, HALF * r.abs() + 2 * HALF * (1 + HALF) * m, "out")
    check_states(final, fin, fmag, "state")


@pytest.mark.parametrize("seed", range(24))
def test_ssm_random_shapes(kda, seed):
    import random
    r = random.Random(seed)
    G = r.choice([1, 2, 3])
    lengths = [r.choice([0, 1, 7, 9, 128, 129, r.randint(1, 500)]) for _ in range(r.randint(1, 7))] if r.random() < 0.5 else None
    if lengths is not None and not sum(lengths):
        lengths[0] = 5
    T = sum(lengths) if lengths is not None else r.choice([r.randint(1, 40), r.randint(100, 900)])
    check_ssm(kda, 1 if lengths is not None else r.randint(1, 4), T, G * r.randint(1, 4), r.choice([64, 128]), G, state=r.choice(["fp32", "bf16"]),
              init=r.random() < 0.6, lengths=lengths, strided=r.random() < 0.5, in_place=r.random() < 0.5, use_D=r.random() < 0.7,
              workspace=r.random() < 0.7, seed=seed, dt_scale=r.choice([1.0, 4.0]))


@pytest.mark.parametrize("seed", range(16))
def test_conv_random_shapes(kda, seed):
    import random
    r = random.Random(seed)
    lengths = [r.choice([0, 1, 2, 3, 63, 64, 65, r.randint(1, 300)]) for _ in range(r.randint(1, 9))] if r.random() < 0.5 else None
    if lengths is not None and not sum(lengths):
        lengths[0] = 2
    T = sum(lengths) if lengths is not None else r.randint(1, 400)
    check_conv(kda, 1 if lengths is not None else r.randint(1, 5), T, 8 * r.choice([1, 5, 31, 32, 33, 70, r.randint(1, 300)]), r.choice([2, 3, 4]),
               silu=r.random() < 0.5, bias=r.random() < 0.5, init=r.random() < 0.6, lengths=lengths, strided=r.random() < 0.5,
               in_place=r.random() < 0.4, seed=seed)


def test_layers_hand_their_states_from_a_prompt_to_steps(kda):
    """examples/hybrid_layers.py: prompts, then single tokens, against one longer prompt. Both are bf16
    models of two layers whose roundings differ along the way: ten roundings of 2^-8 that add as squares."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layers.py")
    spec = importlib.util.spec_from_file_location("hybrid_layers", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main() <= 10 ** 0.5 * HALF
