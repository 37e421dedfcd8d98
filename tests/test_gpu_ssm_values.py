"""GPU tests of what the state-space scan does with special and extreme values: parameters that are
not a number."""
import pytest
import torch

from tests.test_gpu_block import NAN, gen, randn, ssm_inputs

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
