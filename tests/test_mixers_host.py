"""The mixers beside KDA check their arguments on the host and refuse bad calls before any GPU is touched (CPU only): direct
C-ABI calls with dummy, never dereferenced addresses, and the Python calls with CPU tensors."""
import pytest
import torch

from tests.test_block_host import ALIGN, DTYPE, MISMATCH, NULL, RANGE, SHAPE, call, kda  # noqa: F401

NO_GPU = 7  # KDA_ERR_LAUNCH: a call that is not refused gets as far as the missing GPU
without_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would launch with these addresses")

# 16 tokens of 4 value and 2 key heads of 128; rows 0x400 and 0x200 bytes apart
GDN = ("q", "qs", "k", "ks", "v", "vs", "a", "as_", "beta", "bs", "scale", "out", "os", "A", "bias", "init", "idt", "fin", "fdt", "cu", "N", "B",
       "T", "H", "HK", "K", "V", "flags", "stream")
GDN_D = dict(q=0x100000, qs=256, k=0x200000, ks=256, v=0x300000, vs=512, a=0x400000, as_=4, beta=0x500000, bs=4, scale=0.1, out=0x600000, os=512,
             A=0x1000, bias=None, init=None, idt=0, fin=None, fdt=0, cu=None, N=0, B=1, T=16, H=4, HK=2, K=128, V=128, flags=0, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(K=64), SHAPE), (dict(V=64), SHAPE), (dict(H=0), SHAPE), (dict(HK=3), SHAPE), (dict(HK=0), SHAPE), (dict(B=0), SHAPE), (dict(T=-1), SHAPE),
    (dict(cu=0x7000, N=0), SHAPE), (dict(cu=0x7000, N=2, B=2), SHAPE), (dict(T=(1 << 31) - 16), SHAPE), (dict(B=1 << 25, T=1), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(a=None), NULL), (dict(beta=None), NULL), (dict(out=None), NULL),
    (dict(A=None), NULL), (dict(flags=2), RANGE), (dict(flags=9), RANGE), (dict(scale=float("inf")), RANGE), (dict(scale=float("nan")), RANGE),
    (dict(init=0x800000, idt=0), DTYPE), (dict(idt=1), DTYPE), (dict(fin=0x800000, fdt=5), DTYPE),
    (dict(init=0x800000, idt=1, fin=0x8000000, fdt=2), MISMATCH), (dict(init=0x800000, idt=2, fin=0x800400, fdt=2), MISMATCH),
    (dict(qs=248), ALIGN), (dict(ks=252), ALIGN), (dict(vs=500), ALIGN), (dict(os=516), ALIGN), (dict(as_=3), ALIGN), (dict(bs=0), ALIGN),
    (dict(q=0x100008), ALIGN), (dict(out=0x600004), ALIGN), (dict(a=0x400001), ALIGN), (dict(A=0x1002), ALIGN), (dict(fin=0x800008, fdt=2), ALIGN),
    (dict(cu=0x7004, N=1), ALIGN),
    (dict(out=0x300000), MISMATCH), (dict(out=0x100000), MISMATCH), (dict(out=0x200100), MISMATCH), (dict(out=0x400000), MISMATCH),
    (dict(out=0x500000 - 0x10), MISMATCH), (dict(A=0x600000), MISMATCH), (dict(cu=0x600000, N=1), MISMATCH),
    (dict(fin=0x300000, fdt=2), MISMATCH), (dict(fin=0x600000, fdt=1), MISMATCH), (dict(bias=0x800000, fin=0x800000, fdt=2), MISMATCH),
    (dict(init=0x600000, idt=1), MISMATCH),
])
def test_gdn_refusals(kda, over, code):  # noqa: F811
    assert call(kda, "kda_gdn", GDN, GDN_D, over) == code
    assert kda.library().kda_last_error()


@without_gpu
@pytest.mark.parametrize("over", [
    {}, dict(flags=1), dict(init=0x800000, idt=2, fin=0x800000, fdt=2), dict(qs=1024, ks=1024, vs=1024, q=0x100000, k=0x100200, v=0x100400),
    dict(T=4), dict(cu=0x7000, N=3), dict(as_=9, bs=5)])
def test_gdn_calls_that_are_allowed(kda, over):  # noqa: F811
    assert call(kda, "kda_gdn", GDN, GDN_D, over) == NO_GPU


GSTEP = GDN[:15] + ("state", "sdt", "S", "H", "HK", "K", "V", "flags", "stream")
GSTEP_D = {**{k: GDN_D[k] for k in GDN[:15]}, "state": 0x800000, "sdt": 2, "S": 3, "H": 4, "HK": 2, "K": 128, "V": 128, "flags": 0, "stream": None}


@pytest.mark.parametrize("over,code", [
    (dict(S=0), SHAPE), (dict(S=1 << 25), SHAPE), (dict(HK=8), SHAPE), (dict(K=256), SHAPE), (dict(state=None), NULL), (dict(sdt=0), DTYPE),
    (dict(state=0x800004), ALIGN), (dict(flags=4), RANGE), (dict(out=0x300000), MISMATCH), (dict(state=0x300000), MISMATCH),
    (dict(state=0x600000 - 16), MISMATCH), (dict(beta=None), NULL), (dict(vs=100), ALIGN),
])
def test_gdn_step_refusals(kda, over, code):  # noqa: F811
    assert call(kda, "kda_gdn_step", GSTEP, GSTEP_D, over) == code
    assert kda.library().kda_last_error()


QK = ("q", "qs", "k", "ks", "qo", "qos", "ko", "kos", "qw", "kw", "norm", "eps", "pos", "f", "R", "inter", "M", "H", "HK", "D", "stream")
QK_D = dict(q=0x100000, qs=512, k=0x200000, ks=256, qo=0x300000, qos=512, ko=0x400000, kos=256, qw=0x1000, kw=0x2000, norm=1, eps=1e-6, pos=0x3000,
            f=0x4000, R=64, inter=0, M=8, H=4, HK=2, D=128, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(D=96), SHAPE), (dict(D=512), SHAPE), (dict(R=8), SHAPE), (dict(R=144), SHAPE), (dict(R=-16), SHAPE), (dict(H=0), SHAPE), (dict(HK=-1), SHAPE),
    (dict(M=-1), SHAPE), (dict(q=None), NULL), (dict(qo=None), NULL), (dict(k=None), NULL), (dict(ko=None), NULL), (dict(pos=None), NULL),
    (dict(f=None), NULL), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE),
    (dict(qs=504), ALIGN), (dict(ks=252), ALIGN), (dict(qos=508), ALIGN), (dict(kos=128), ALIGN), (dict(q=0x100008), ALIGN), (dict(ko=0x400004), ALIGN),
    (dict(qw=0x1008), ALIGN), (dict(pos=0x3004), ALIGN), (dict(f=0x4002), ALIGN),
    (dict(qo=0x100400), MISMATCH), (dict(qo=0x200000), MISMATCH), (dict(ko=0x100000), MISMATCH), (dict(ko=0x200200), MISMATCH),
    (dict(ko=0x300000), MISMATCH), (dict(qo=0x1000 - 0x10), MISMATCH), (dict(pos=0x300000), MISMATCH), (dict(f=0x400100), MISMATCH),
])
def test_qk_rope_refusals(kda, over, code):  # noqa: F811
    assert call(kda, "kda_qk_rope", QK, QK_D, over) == code
    assert kda.library().kda_last_error()


@without_gpu
@pytest.mark.parametrize("over", [
    {}, dict(qo=0x100000, ko=0x200000), dict(HK=0, k=None, ko=None), dict(R=0, f=None), dict(norm=0, eps=-1.0, qw=None),
    dict(qs=1024, ks=1024, q=0x100000, k=0x100400)])
def test_qk_rope_calls_that_are_allowed(kda, over):  # noqa: F811
    assert call(kda, "kda_qk_rope", QK, QK_D, over) == NO_GPU


def test_no_tokens_need_no_gpu(kda):  # noqa: F811
    assert call(kda, "kda_qk_rope", QK, QK_D, dict(M=0)) == 0
    assert call(kda, "kda_kv_append", APP, APP_D, dict(T=0)) == 0


# 10 pages of 2 heads x 16 tokens of 64 channels, keys and values side by side: pages 0x2000 bytes apart
APP = ("k", "ks", "v", "vs", "kc", "vc", "ps", "pages", "size", "table", "width", "pos", "f", "R", "inter", "kw", "norm", "eps", "cu", "N", "B", "T", "HK",
       "D", "stream")
APP_D = dict(k=0x100000, ks=256, v=0x100100, vs=256, kc=0x200000, vc=0x201000, ps=4096, pages=10, size=16, table=0x1000, width=4, pos=0x2000, f=0x3000,
             R=32, inter=0, kw=0x4000, norm=1, eps=1e-6, cu=None, N=0, B=2, T=8, HK=2, D=64, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(size=12), SHAPE), (dict(size=4), SHAPE), (dict(size=8192), SHAPE), (dict(pages=0), SHAPE), (dict(width=0), SHAPE), (dict(HK=0), SHAPE),
    (dict(D=32), SHAPE), (dict(R=40), SHAPE), (dict(B=0), SHAPE), (dict(cu=0x7000, N=1), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(table=None), NULL), (dict(pos=None), NULL), (dict(f=None), NULL), (dict(eps=float("inf")), RANGE),
    (dict(ks=120), ALIGN), (dict(vs=132), ALIGN), (dict(ps=2040), ALIGN), (dict(ps=4100), ALIGN), (dict(kc=0x200008), ALIGN), (dict(table=0x1002), ALIGN),
    (dict(pos=0x2004), ALIGN), (dict(kw=0x4004), ALIGN), (dict(k=0x100008), ALIGN),
    (dict(vc=0x200000), MISMATCH), (dict(vc=0x200800), MISMATCH), (dict(k=0x200000), MISMATCH), (dict(v=0x201000), MISMATCH), (dict(table=0x203000), MISMATCH),
    (dict(pos=0x202000), MISMATCH), (dict(kw=0x201010), MISMATCH), (dict(f=0x200010), MISMATCH), (dict(cu=0x200008, N=1, B=1), MISMATCH),
])
def test_kv_append_refusals(kda, over, code):  # noqa: F811
    assert call(kda, "kda_kv_append", APP, APP_D, over) == code
    assert kda.library().kda_last_error()


@without_gpu
@pytest.mark.parametrize("over", [{}, dict(R=0, f=None, norm=0, kw=None), dict(cu=0x7000, N=3, B=1), dict(vc=0x800000, ps=2048)])
def test_kv_append_calls_that_are_allowed(kda, over):  # noqa: F811
    assert call(kda, "kda_kv_append", APP, APP_D, over) == NO_GPU


ATT = ("q", "qs", "kc", "vc", "ps", "pages", "size", "table", "width", "pos", "scale", "out", "os", "lse", "S", "H", "HK", "D", "ws", "wsb", "stream")
ATT_D = dict(q=0x100000, qs=256, kc=0x200000, vc=0x201000, ps=4096, pages=10, size=16, table=0x1000, width=4, pos=0x2000, scale=0.1, out=0x300000, os=256,
             lse=0x3000, S=3, H=4, HK=2, D=64, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(S=0), SHAPE), (dict(S=1 << 17), SHAPE), (dict(H=3), SHAPE), (dict(HK=0), SHAPE), (dict(D=256), SHAPE), (dict(size=24), SHAPE), (dict(pages=-1), SHAPE),
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(pos=None), NULL), (dict(kc=None), NULL), (dict(table=None), NULL), (dict(scale=float("nan")), RANGE),
    (dict(qs=252), ALIGN), (dict(os=248), ALIGN), (dict(q=0x100004), ALIGN), (dict(lse=0x3002), ALIGN), (dict(ws=0x400008, wsb=64), ALIGN),
    (dict(pos=0x2001), ALIGN), (dict(ps=1000), ALIGN),
    (dict(out=0x100000), MISMATCH), (dict(out=0x200000), MISMATCH), (dict(out=0x1000 - 16), MISMATCH), (dict(lse=0x300000), MISMATCH),
    (dict(lse=0x100010), MISMATCH), (dict(lse=0x201000), MISMATCH), (dict(lse=0x2000), MISMATCH),
])
def test_attn_step_refusals(kda, over, code):  # noqa: F811
    assert call(kda, "kda_attn_step", ATT, ATT_D, over) == code
    assert kda.library().kda_last_error()


def test_attn_step_workspace_refusals(kda):  # noqa: F811
    import ctypes
    n = ctypes.c_size_t(7)
    f = kda.library().kda_attn_step_workspace_bytes
    assert f(1, 4, 2, 64, None) == NULL
    for bad in ((-1, 4, 2, 64), (1, 3, 2, 64), (1, 4, 0, 64), (1, 4, 2, 96)):
        assert f(*bad, ctypes.byref(n)) == SHAPE
    assert n.value == 7


def test_python_calls_refuse_bad_tensors(kda):  # noqa: F811
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="v must be a CUDA tensor"):
        kda.gdn(x, x, x, x[..., 0], x[..., 0], 1.0, x, torch.zeros(2))
    with pytest.raises(ValueError, match=r"v must be \[B, T, H, 128\]"):
        kda.gdn(x, x, x[0], x[..., 0], x[..., 0], 1.0, x, torch.zeros(2))
    with pytest.raises(ValueError, match=r"v must be \[S, H, 128\]"):
        kda.gdn_step(x, x, x, x, x, 1.0, x, None, None)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kda.qk_rope(x, None, x, None, torch.zeros(1, 4, dtype=torch.int64))
    with pytest.raises(ValueError, match="k must be"):
        kda.kv_append("rows", x, x, x, x, x)
    with pytest.raises(ValueError, match=r"q must be \[S, H, D\]"):
        kda.attn_step(x, x, x, x, x, x, 1.0)


def test_python_page_checks_name_the_argument(kda):  # noqa: F811
    from gated_linear_attention_kda_gb300 import mixers
    c = torch.zeros(6, 2, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    dev = c.get_device()  # a CPU tensor's own "device index": the layout checks run as they would on a GPU
    got = mixers._pages(c[:, 0], c[:, 1], table, 3, 2, 64, dev)
    assert got[2:5] == (c.stride(0), 6, 16) and got[6] == 4
    with pytest.raises(ValueError, match="v_cache: the elements of one page must be contiguous"):
        mixers._pages(c[:, 0], c[:, 1].transpose(1, 2).contiguous().transpose(1, 2), table, 3, 2, 64, dev)
    with pytest.raises(ValueError, match="same page stride"):
        mixers._pages(c[:, 0], c[:, 1].contiguous(), table, 3, 2, 64, dev)
    with pytest.raises(ValueError, match="page_table"):
        mixers._pages(c[:, 0], c[:, 1], table[:2].float(), 3, 2, 64, dev)
    with pytest.raises(ValueError, match=r"k_cache must be \[pages"):
        mixers._pages(c, c, table, 3, 2, 64, dev)
