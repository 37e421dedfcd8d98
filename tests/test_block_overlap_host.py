"""What the operators around the mixer write shares no memory with anything else that a call names, but for
the pairs that an entry point allows: refused on the host before any GPU is touched (CPU only; dummy
addresses that are never dereferenced). Where nothing is refused, the call gets as far as the missing GPU."""
import pytest

from tests.test_block_host import CONV, CONV_D, GATED, GATED_D, MISMATCH, RES, RES_D, SSM, SSM_D, SSTEP, SSTEP_D, STEP, STEP_D, call, kda  # noqa: F401

NO_GPU = 7  # KDA_ERR_LAUNCH


@pytest.fixture(autouse=True)
def no_gpu():
    """A call that is not refused would launch with these addresses."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")


# state bytes: conv 1 x 3 x 64 bf16 (384), ssm 4 x 64 x 128 fp32 (131,072)
@pytest.mark.parametrize("over", [
    dict(fin=0x100000), dict(fin=0x100000 + 16 * 128 - 16),       # x: its first row, the end of its last
    dict(fin=0x900000), dict(fin=0x900000 - 368),                 # out, by the last 16 bytes
    dict(fin=0x1000), dict(fin=0x1000 + 1008), dict(b=0x2000, fin=0x2000),
    dict(fin=0x7000, cu=0x7000, N=1), dict(init=0x900000), dict(init=0x900400, fin=0x300000),
    dict(out=0x1000), dict(b=0x900100), dict(cu=0x900008, N=1),
])
def test_conv(kda, over):  # noqa: F811
    assert call(kda, "kda_conv", CONV, CONV_D, over) == MISMATCH
    assert kda.library().kda_last_error()


@pytest.mark.parametrize("over", [dict(state=0x100000), dict(state=0x900000 + 4 * 128 - 16), dict(state=0x1000), dict(b=0x500100), dict(out=0x1000)])
def test_conv_step(kda, over):  # noqa: F811
    assert call(kda, "kda_conv_step", STEP, STEP_D, over) == MISMATCH


@pytest.mark.parametrize("over", [
    dict(fin=0x100000, fdt=2), dict(fin=0x100000 - 131056, fdt=2), dict(fin=0x200000, fdt=1), dict(fin=0x300000, fdt=2), dict(fin=0x400000, fdt=1),
    dict(fin=0x500000, fdt=2), dict(fin=0x4e0010, fdt=2), dict(fin=0x1000, fdt=2), dict(D=0x800100, fin=0x800000, fdt=2),
    dict(bias=0x800100, fin=0x800000, fdt=2), dict(cu=0x800008, N=1, fin=0x800000, fdt=2), dict(init=0x500000, idt=2),
    dict(init=0x501ff0, idt=1, fin=0x900000, fdt=1), dict(A=0x500004), dict(D=0x500ffc), dict(cu=0x500000, N=1),
])
def test_ssm(kda, over):  # noqa: F811
    assert call(kda, "kda_ssm", SSM, SSM_D, over) == MISMATCH
    assert kda.library().kda_last_error()


@pytest.mark.parametrize("over", [
    dict(state=0x100000), dict(state=0x200000), dict(state=0x300000, sdt=1), dict(state=0x400000), dict(state=0x500000), dict(state=0x4a0010),
    dict(A=0x800000), dict(D=0x800100), dict(bias=0x500000),
])
def test_ssm_step(kda, over):  # noqa: F811
    assert call(kda, "kda_ssm_step", SSTEP, SSTEP_D, over) == MISMATCH


@pytest.mark.parametrize("fn,names,defaults,over", [
    ("kda_gated_norm", GATED, GATED_D, dict(w=0x300100)), ("kda_gated_norm", GATED, GATED_D, dict(out=0x1000)),
    ("kda_residual_norm", RES, RES_D, dict(w=0x400000)), ("kda_residual_norm", RES, RES_D, dict(pw=0x300000)),
    ("kda_residual_norm", RES, RES_D, dict(ch=0x400200)),
])
def test_norms(kda, fn, names, defaults, over):  # noqa: F811
    assert call(kda, fn, names, defaults, over) == MISMATCH


@pytest.mark.parametrize("fn,names,defaults,over", [
    # states in place, and right behind or between other buffers
    ("kda_conv", CONV, CONV_D, dict(init=0x200000, fin=0x200000)), ("kda_conv", CONV, CONV_D, dict(fin=0x100000 + 16 * 128)),
    ("kda_conv", CONV, CONV_D, dict(fin=0x900000 - 384)), ("kda_conv", CONV, CONV_D, dict(xs=1024, fin=0x100000 + 128)),
    ("kda_conv", CONV, CONV_D, dict(xs=1024, fin=0x100000 + 7 * 2048 + 128)),
    ("kda_ssm", SSM, SSM_D, dict(init=0x800000, idt=2, fin=0x800000, fdt=2)), ("kda_ssm", SSM, SSM_D, dict(fin=0x100000 - 131072, fdt=2)),
    ("kda_ssm", SSM, SSM_D, dict(fin=0x500000 + 16 * 512, fdt=2)), ("kda_ssm", SSM, SSM_D, dict(init=0x100000, idt=2)),
    ("kda_conv_step", STEP, STEP_D, dict(out=0x100000)), ("kda_ssm_step", SSTEP, SSTEP_D, dict(state=0x500000 + 3 * 512)),
    ("kda_gated_norm", GATED, GATED_D, dict(out=0x100000)), ("kda_residual_norm", RES, RES_D, dict(ro=0x200000, out=0x100000)),
])
def test_what_is_allowed(kda, fn, names, defaults, over):  # noqa: F811
    assert call(kda, fn, names, defaults, over) == NO_GPU
