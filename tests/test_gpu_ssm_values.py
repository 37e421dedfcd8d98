"""GPU tests of what the state-space scan does with special and extreme values: parameters and
states that hold no number, a skip term far above the scan's own terms, x that holds NaN or infinity.

Tolerances as in tests/test_gpu_block.py, with one difference where a test says so: the bound on an
output's own rounding is half a step at that value, not 2^-8 of it, and the skip term D x carries no
rounding but that one (fp32 arithmetic: 2^-22 of it)."""
import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_block import HALF, NAN, close, gen, randn, ssm_inputs

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def kda():
    import gated_linear_attention_kda_gb300 as m
    return m


def workspace_of(kda, S, tokens, H, P):
    return torch.empty(kda.ssm_workspace_bytes(S, tokens, H, P), dtype=torch.uint8, device="cuda")


# 5 and 8 tokens run token by token, 9 to 300 in chunks, 1500 cut along time where there is a workspace
LENGTHS = [5, 8, 9, 128, 300, 1500]


@pytest.mark.parametrize("which", ["A_log", "dt_bias", "D"])
@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("P", [64, 128])
def test_a_parameter_that_is_not_a_number_leaves_no_number_in_its_head(kda, which, T, P):
    g = gen(T + P)
    args = dict(zip(("x", "dt", "b", "c", "A_log", "D", "dt_bias"), (v.clone() for v in ssm_inputs(g, 1, T, 2, P, 1))))
    init = randn(g, 1, 2, P, 128, dtype=torch.float32)
    ws = workspace_of(kda, 1, T, 2, P)
    assert (ws.numel() > 0) == (T == 1500)

    def run():
        out, fin = torch.full((1, T, 2, P), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full_like(init, 7.0)
        kda.ssm(out=out, initial_state=init, final_state=fin, workspace=ws, **args)
        kda.check_device_status()
        return out, fin

    ref, ref_fin = run()
    args[which][1] = NAN
    out, fin = run()
    assert torch.equal(out[:, :, 0], ref[:, :, 0]) and torch.equal(fin[:, 0], ref_fin[:, 0])
    assert torch.isnan(out[:, :, 1]).all()
    if which == "D":
        assert torch.equal(fin, ref_fin)
    else:
        assert torch.isnan(fin[:, 1]).all()


def half_step(ref, mantissa_bits=8):
    """Half a bf16 step at each value."""
    return 2.0 ** (torch.floor(torch.log2(ref.abs().clamp_min(2.0 ** -120))) - mantissa_bits)


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("use_workspace", [False, True])
def test_the_skip_term_keeps_its_32_bits(kda, T, P, use_workspace):
    """D far above the scan's terms and with more bits than bf16 has: outputs are D x and the scan's sum, rounded once."""
    g = gen(T + P)
    x, dt, b, c, A_log, _, dt_bias = ssm_inputs(g, 2, T, 3, P, 1)
    b, c = b * 0.125, c * 0.125
    D = torch.tensor([100.24609375, -3.0107421875, 0.3330078125], device="cuda")
    ref, _, mag, _ = R.ssm(x, dt, b, c, A_log, None, dt_bias, None)
    skip = D.double()[:, None] * x.double()
    out = torch.full((2, T, 3, P), NAN, dtype=torch.bfloat16, device="cuda")
    kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, workspace=workspace_of(kda, 2, 2 * T, 3, P) if use_workspace else None)
    kda.check_device_status()
    ref = ref + skip
    # ahead of the last rounding: the scan's own slack, and fp32 sums of the skip term; a value near a power of two may
    # round on the far side of it, where a step is twice as long
    ahead = 2 * HALF * (1 + HALF) * mag + 2.0 ** -22 * skip.abs()
    close(out, ref, ahead + half_step(ref.abs() + ahead) + 1e-30, "out")


def spoil_and_compare(kda, x, dt, b, c, A_log, D, dt_bias, init, spots, bad, lengths=None, ws=None, fin=True, in_place=False):
    """Run with ``bad`` in x at ``spots`` (token of the packed axis, head, channel): what lies ahead of the first spot of its
    sequence, head and channel is what the recurrence gives, what lies behind holds no number; every other channel is bit
    for bit what it is without. ``init`` is kept."""
    B, T, H, P = x.shape
    cu = torch.tensor([0] + list(lengths)).cumsum(0).cuda() if lengths is not None else None
    S = len(lengths) if lengths is not None else B
    spans = R.spans(B, T, cu)

    def run(x):
        first = init.clone() if init is not None else None
        final = (first if in_place else torch.full((S, H, P, 128), 7.0, device="cuda")) if fin else None
        out = torch.full((B, T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, initial_state=first, final_state=final, cu_seqlens=cu, workspace=ws)
        kda.check_device_status()
        return out.view(B * T, H, P), final

    clean, clean_fin = run(x)
    ref, _, mag, _ = R.ssm(x, dt, b, c, A_log, D, dt_bias, init, cu)
    ref, mag = ref.view(B * T, H, P), mag.view(B * T, H, P)
    spoilt = x.clone()
    for t, h, p in spots:
        spoilt.view(B * T, H, P)[t, h, p] = bad
    out, final = run(spoilt)
    behind = torch.zeros(B * T, H, P, dtype=torch.bool, device="cuda")
    touched, channels = behind.clone(), torch.zeros(S, H, P, dtype=torch.bool, device="cuda")
    for t, h, p in spots:
        s = next(i for i, (s0, s1) in enumerate(spans) if s0 <= t < s1)
        behind[t:spans[s][1], h, p] = True
        touched[spans[s][0]:spans[s][1], h, p] = True
        channels[s, h, p] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert not torch.isfinite(out[behind]).any()
    ahead = touched & ~behind
    r, m = ref[ahead], mag[ahead]
    close(out[ahead], r, HALF * r.abs() + 2 * HALF * (1 + HALF) * m + 1e-30, "ahead")
    if fin:
        assert torch.equal(final[~channels], clean_fin[~channels]) and not torch.isfinite(final[channels]).any()


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("T,at", [(9, 8), (128, 127), (300, 200), (300, 256), (300, 299), (400, 130), (1500, 1000), (1500, 0)])
@pytest.mark.parametrize("cut", [False, True])
def test_a_non_finite_x_leaves_earlier_tokens_alone(kda, P, T, at, bad, cut):
    g = gen(T + at)
    args = [v.clone() for v in ssm_inputs(g, 1, T, 2, P, 1)]
    args[4] -= 6  # weak decay: what was spoilt stays
    ws = workspace_of(kda, 1, T, 2, P) if cut else None
    assert not cut or (ws.numel() > 0) == (T == 1500)
    spoil_and_compare(kda, *args, randn(g, 1, 2, P, 128, dtype=torch.float32), [(at, 1, 9)], bad, ws=ws)


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cut", [False, True])
def test_many_non_finite_channels_of_packed_sequences(kda, P, in_place, cut):
    """Several channels and tokens of some sequences, two heads, states in place; the first and last channel among them."""
    g = gen(P)
    lengths = [200, 1, 0, 2900, 3500, 129]
    T = sum(lengths)
    args = [v.clone() for v in ssm_inputs(g, 1, T, 2, P, 1)]
    args[4] -= 6
    spots = [(150, 0, 0), (150, 0, P - 1), (30, 0, P - 1), (200, 1, 5), (201 + 2899, 1, 33), (3101 + 700, 0, 31), (3101 + 1400, 0, 31),
             (6601 + 128, 1, 63)] + [(3101 + 260 + p, 1, p) for p in range(P)]
    ws = workspace_of(kda, len(lengths), T, 2, P) if cut else None
    assert not cut or ws.numel() > 0
    spoil_and_compare(kda, *args, randn(g, len(lengths), 2, P, 128, dtype=torch.float32), spots, NAN, lengths=lengths, ws=ws, in_place=in_place)


@pytest.mark.parametrize("P", [64, 128])
def test_non_finite_x_without_states_or_skip(kda, P):
    """No initial and no final state, no D: what is written is the outputs alone."""
    g = gen(P + 1)
    args = [v.clone() for v in ssm_inputs(g, 3, 333, 2, P, 2)]
    args[4] -= 6
    args[5] = None
    spoil_and_compare(kda, *args, None, [(100, 0, 3), (333 + 290, 1, 17), (666 + 332, 1, 40)], NAN, fin=False)


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("bad", [NAN, INF])
def test_an_initial_state_that_holds_no_number_stays_in_its_channel(kda, T, state, bad):
    g = gen(T)
    x, dt, b, c, A_log, D, dt_bias = (v.clone() for v in ssm_inputs(g, 1, T, 2, 64, 1))
    A_log -= 6
    init = randn(g, 1, 2, 64, 128, dtype=state)
    ws = workspace_of(kda, 1, T, 2, 64)

    def run():
        out, fin = torch.full((1, T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full_like(init, 7.0)
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, initial_state=init, final_state=fin, workspace=ws)
        kda.check_device_status()
        return out, fin

    ref, ref_fin = run()
    init[0, 1, 20, 77] = bad
    out, fin = run()
    assert not torch.isfinite(out[0, :, 1, 20]).any() and not torch.isfinite(fin[0, 1, 20, 77])
    rest, cell = torch.ones_like(out, dtype=torch.bool), torch.ones_like(fin, dtype=torch.bool)
    rest[0, :, 1, 20] = False
    cell[0, 1, 20, 77] = False
    assert torch.equal(out[rest], ref[rest]) and torch.equal(fin[cell], ref_fin[cell])
