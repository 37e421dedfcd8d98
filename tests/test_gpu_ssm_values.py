"""GPU tests of what the state-space scan does with special and extreme values: parameters that
are not a number, a skip term far above the scan's own terms.

Tolerances as in tests/test_gpu_block.py, with one difference where a test says so: the bound on an
output's own rounding is half a step at that value, not 2^-8 of it, and the skip term D x carries no
rounding but that one (fp32 arithmetic: 2^-22 of it)."""
import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_block import HALF, NAN, close, gen, randn, ssm_inputs

pytestmark = pytest.mark.gpu


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
