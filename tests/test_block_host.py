"""The operators around the mixer check their arguments on the host and refuse bad calls before any
GPU is touched (CPU only): direct C-ABI calls with dummy, never dereferenced addresses, and the
Python calls with CPU tensors."""
import ctypes

import pytest
import torch

NULL, SHAPE, DTYPE, RANGE, MISMATCH, ALIGN = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__
    __graft_entry__._builder().build_library()
    import gated_linear_attention_kda_gb300 as m
    return m


def call(kda, fn, names, defaults, over):
    args = dict(defaults)
    assert set(over) <= set(args), over
    args.update(over)
    return getattr(kda.library(), fn)(*[args[n] for n in names])


CONV = ("x", "xs", "w", "b", "act", "out", "os", "init", "fin", "cu", "N", "B", "T", "C", "W", "stream")
CONV_D = dict(x=0x100000, xs=64, w=0x1000, b=None, act=2, out=0x900000, os=64, init=None, fin=None, cu=None, N=0, B=1, T=16, C=64, W=4,
              stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(W=1), SHAPE), (dict(W=5), SHAPE), (dict(C=60), SHAPE), (dict(C=0), SHAPE), (dict(B=0), SHAPE), (dict(T=-1), SHAPE),
    (dict(cu=0x7000, B=2, N=1), SHAPE), (dict(cu=0x7000, N=0), SHAPE), (dict(B=1 << 20, T=1 << 12), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(act=1), RANGE), (dict(act=7), RANGE),
    (dict(xs=56), ALIGN), (dict(xs=68), ALIGN), (dict(os=60), ALIGN), (dict(x=0x100008), ALIGN), (dict(out=0x900004), ALIGN),
    (dict(w=0x1008), ALIGN), (dict(b=0x1004), ALIGN), (dict(fin=0x2008), ALIGN), (dict(cu=0x7004, N=1), ALIGN),
    (dict(out=0x100000), MISMATCH), (dict(out=0x100080), MISMATCH),          # the same rows, and rows shifted by one token
    (dict(xs=192, os=192, out=0x100000 + 64), MISMATCH),                      # slices of one row that share channels
    (dict(init=0x200000, fin=0x200010), MISMATCH),
])
def test_conv_refusals(kda, over, code):
    assert call(kda, "kda_conv", CONV, CONV_D, over) == code
    assert kda.library().kda_last_error()


STEP = ("x", "xs", "w", "b", "act", "out", "os", "state", "S", "C", "W", "stream")
STEP_D = dict(x=0x100000, xs=64, w=0x1000, b=None, act=2, out=0x900000, os=64, state=0x500000, S=4, C=64, W=4, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(S=0), SHAPE), (dict(W=6), SHAPE), (dict(C=4), SHAPE), (dict(state=None), NULL), (dict(x=None), NULL),
    (dict(state=0x500008), ALIGN), (dict(xs=60), ALIGN), (dict(act=3), RANGE),
    (dict(out=0x100080), MISMATCH), (dict(out=0x100000, os=128), MISMATCH),  # out may be x itself, not its shifted rows
])
def test_conv_step_refusals(kda, over, code):
    assert call(kda, "kda_conv_step", STEP, STEP_D, over) == code


SSM = ("x", "xs", "dt", "dts", "b", "bs", "c", "cs", "A", "D", "bias", "out", "os", "init", "idt", "fin", "fdt", "cu", "N", "B", "T", "H", "P",
       "G", "K", "ws", "wsb", "stream")
SSM_D = dict(x=0x100000, xs=256, dt=0x200000, dts=4, b=0x300000, bs=128, c=0x400000, cs=128, A=0x1000, D=None, bias=None, out=0x500000, os=256,
             init=None, idt=0, fin=None, fdt=0, cu=None, N=0, B=1, T=16, H=4, P=64, G=1, K=128, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(P=32), SHAPE), (dict(P=256), SHAPE), (dict(K=64), SHAPE), (dict(H=0), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE),
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(cu=0x7000, N=0), SHAPE), (dict(cu=0x7000, N=2, B=2), SHAPE),
    (dict(T=(1 << 31) - 16), SHAPE), (dict(B=1 << 25, T=1, H=4), SHAPE),
    (dict(x=None), NULL), (dict(dt=None), NULL), (dict(b=None), NULL), (dict(c=None), NULL), (dict(out=None), NULL), (dict(A=None), NULL),
    (dict(init=0x800000, idt=0), DTYPE), (dict(idt=1), DTYPE), (dict(fin=0x800000, fdt=5), DTYPE),
    (dict(init=0x800000, idt=1, fin=0x8000000, fdt=2), MISMATCH), (dict(init=0x800000, idt=2, fin=0x800400, fdt=2), MISMATCH),
    (dict(out=0x100000), MISMATCH), (dict(out=0x300000), MISMATCH), (dict(out=0x200000), MISMATCH),
    (dict(xs=248), ALIGN), (dict(os=260), ALIGN), (dict(bs=100), ALIGN), (dict(dts=3), ALIGN), (dict(x=0x100008), ALIGN),
    (dict(dt=0x200001), ALIGN), (dict(A=0x1002), ALIGN), (dict(fin=0x800008, fdt=2), ALIGN), (dict(ws=0x900008, wsb=64), ALIGN),
    (dict(cu=0x7004, N=1), ALIGN),
])
def test_ssm_refusals(kda, over, code):
    assert call(kda, "kda_ssm", SSM, SSM_D, over) == code
    assert kda.library().kda_last_error()


SSTEP = SSM[:13] + ("state", "sdt", "S", "H", "P", "G", "K", "stream")
SSTEP_D = {**{k: SSM_D[k] for k in SSM[:13]}, "state": 0x800000, "sdt": 2, "S": 3, "H": 4, "P": 64, "G": 1, "K": 128, "stream": None}


@pytest.mark.parametrize("over,code", [
    (dict(S=0), SHAPE), (dict(P=96), SHAPE), (dict(K=256), SHAPE), (dict(G=8), SHAPE), (dict(state=None), NULL), (dict(sdt=0), DTYPE),
    (dict(state=0x800004), ALIGN), (dict(out=0x100000), MISMATCH), (dict(c=None), NULL),
])
def test_ssm_step_refusals(kda, over, code):
    assert call(kda, "kda_ssm_step", SSTEP, SSTEP_D, over) == code


GATED = ("x", "xs", "z", "zs", "w", "wr", "out", "os", "eps", "act", "first", "M", "R", "D", "stream")
GATED_D = dict(x=0x100000, xs=256, z=0x200000, zs=256, w=0x1000, wr=1, out=0x300000, os=256, eps=1e-5, act=1, first=0, M=8, R=2, D=128, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(D=12), SHAPE), (dict(D=16392), SHAPE), (dict(R=0), SHAPE), (dict(M=-1), SHAPE), (dict(wr=3), SHAPE),
    (dict(x=None), NULL), (dict(z=None), NULL), (dict(out=None), NULL),
    (dict(act=3), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE),
    (dict(xs=250), ALIGN), (dict(zs=128), ALIGN), (dict(w=0x1004), ALIGN), (dict(out=0x300008), ALIGN),
    (dict(out=0x100100), MISMATCH), (dict(out=0x200000, os=512), MISMATCH),
])
def test_gated_norm_refusals(kda, over, code):
    assert call(kda, "kda_gated_norm", GATED, GATED_D, over) == code


RES = ("x", "xs", "r", "rs", "ro", "ros", "rdt", "z", "zs", "act", "pw", "ch", "alpha", "w", "out", "os", "eps", "M", "D", "stream")
RES_D = dict(x=0x100000, xs=256, r=0x200000, rs=256, ro=0x300000, ros=256, rdt=2, z=None, zs=256, act=0, pw=None, ch=None, alpha=1.0, w=None,
             out=0x400000, os=256, eps=1e-5, M=8, D=256, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(D=4), SHAPE), (dict(D=20000), SHAPE), (dict(M=-1), SHAPE), (dict(rdt=0), DTYPE), (dict(rdt=3), DTYPE),
    (dict(x=None), NULL), (dict(r=None), NULL), (dict(ro=None, out=None), NULL),
    (dict(act=9), RANGE), (dict(eps=float("inf")), RANGE), (dict(alpha=float("nan")), RANGE),
    (dict(rs=250), ALIGN), (dict(rs=128), ALIGN), (dict(xs=252), ALIGN), (dict(pw=0x1008), ALIGN), (dict(r=0x200004), ALIGN),
    (dict(ro=0x100000), MISMATCH), (dict(out=0x200000), MISMATCH), (dict(ro=0x200400), MISMATCH), (dict(out=0x300000), MISMATCH),
    (dict(z=0x300000), MISMATCH),
])
def test_residual_norm_refusals(kda, over, code):
    assert call(kda, "kda_residual_norm", RES, RES_D, over) == code


def test_empty_norms_are_no_work(kda):
    assert call(kda, "kda_gated_norm", GATED, GATED_D, dict(M=0)) == 0
    assert call(kda, "kda_residual_norm", RES, RES_D, dict(M=0)) == 0


def test_workspace_query_refusals(kda):
    lib = kda.library()
    n = ctypes.c_size_t(7)
    assert lib.kda_ssm_workspace_bytes(1, 1, 1, 64, None) == NULL
    for bad in ((-1, 1, 1, 64), (1, -1, 1, 64), (1, 1, 0, 64), (1, 1, 1, 32)):
        assert lib.kda_ssm_workspace_bytes(*bad, ctypes.byref(n)) == SHAPE
    assert n.value == 7


def test_python_calls_refuse_bad_tensors(kda):
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 4)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.conv(x, w, x.clone())
    with pytest.raises(ValueError, match=r"x must be \[B, T, C\]"):
        kda.conv(x[0], w, x[0].clone())
    with pytest.raises(ValueError, match=r"x must be \[S, C\]"):
        kda.conv_step(x, w, x.clone(), x)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.residual_norm(x, x, None, out=x.clone())
    h = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.gated_norm(h, h, None, h.clone())
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.ssm(h, h[..., 0], h, h, h.clone(), torch.zeros(2))
    with pytest.raises(ValueError, match=r"x must be \[S, H, P\]"):
        kda.ssm_step(h, h, h, h, h, None, None)
    with pytest.raises(ValueError, match="x must be"):
        kda.gated_norm("rows", h, None, h)


def test_python_argument_checks_name_the_argument(kda):
    """The checks below the device check, on CPU tensors through the helpers the calls share."""
    from gated_linear_attention_kda_gb300 import block
    t = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="gate must be a torch.Tensor"):
        block._rows("gate", [1.0], t.shape, 2, 0)
    with pytest.raises(ValueError, match="gate must be a CUDA tensor"):
        block._rows("gate", t, t.shape, 2, 0)
    dev = t.get_device()  # a CPU tensor's own "device index": the layout checks run as they would on a GPU
    with pytest.raises(ValueError, match="elements of one token must be contiguous"):
        block._rows("x", torch.zeros(2, 3, 16, dtype=torch.bfloat16)[..., ::2], (2, 3, 8), 2, dev)
    with pytest.raises(ValueError, match="batch rows must follow one another"):
        block._rows("x", torch.zeros(2, 5, 8, dtype=torch.bfloat16)[:, :3], (2, 3, 8), 2, dev)
    assert block._rows("x", torch.zeros(2, 3, 32, dtype=torch.bfloat16)[..., 8:16], (2, 3, 8), 2, dev)[1] == 32
    assert block._rows("x", torch.zeros(2, 1, 8, dtype=torch.bfloat16), (2, 1, 8), 2, dev)[1] == 8
    with pytest.raises(ValueError, match="must be contiguous"):
        block._dense("weight", torch.zeros(4, 64).T, dev, (torch.float32,), (64, 4))
    with pytest.raises(ValueError, match="act must be one of"):
        block._act("relu")
