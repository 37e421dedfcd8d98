"""The operators around the mixer: short causal convolution, selective state-space scan, gated norm
and residual norm, for prompts and for single tokens (``include/kda.h``, "Operators around the
mixer"). Argument marshalling only, as in the package's other calls: every function writes the
buffers it is given on the current CUDA stream, allocates nothing and returns them.

Token axes may be strided: a slice of a projection's row is passed as it stands. The elements of
one token are contiguous, and batch rows follow one another at the token stride.

The checks read each tensor's properties once and the calls pass plain integers: for a single
token the host's time is the call's time (a call costs 8 to 16 us of it on the GB300's CPU).
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE_BF16, DTYPE_FP32, DTYPE_NONE, _lib, _P, _F, _I, _I64, _raise

_Z = ctypes.c_size_t
_BF16, _F32 = torch.bfloat16, torch.float32
_CODES = {_BF16: DTYPE_BF16, _F32: DTYPE_FP32}
ACTS = {"none": 0, "sigmoid": 1, "silu": 2}  # KDA_ACT_*

_lib.kda_conv.argtypes = [_P, _I64, _P, _P, _I, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_conv_step.argtypes = [_P, _I64, _P, _P, _I, _P, _I64, _P, _I64, _I64, _I64, _P]
_lib.kda_ssm.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _I, _P, _I, _P,
                         _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P, _Z, _P]
_lib.kda_ssm_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, ctypes.POINTER(_Z)]
_lib.kda_ssm_step.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _I,
                              _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_gated_norm.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _F, _I, _I, _I64, _I64, _I64, _P]
_lib.kda_residual_norm.argtypes = [_P, _I64, _P, _I64, _P, _I64, _I, _P, _I64, _I, _P, _P, _F, _P, _P, _I64, _F,
                                   _I64, _I64, _P]
for _f in ("kda_conv", "kda_conv_step", "kda_ssm", "kda_ssm_workspace_bytes", "kda_ssm_step", "kda_gated_norm",
           "kda_residual_norm"):
    getattr(_lib, _f).restype = _I


def _refuse(name, t, dev, dtypes, shape):
    """Say what is wrong with a tensor's kind, device, type or shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but x is on cuda:{dev}: all tensors must share one device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _x_device(x, dims, layout):
    """The device of the leading argument, whose shape the others are checked against."""
    if not isinstance(x, torch.Tensor) or x.dim() not in dims:
        raise ValueError(f"x must be {layout}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    return x.get_device()


def _rows(name, t, shape, lead, dev, dtypes=(_BF16,)):
    """Check an activation of the given shape; returns its address and the distance in elements
    between its tokens. The first ``lead`` dimensions are the token axes ([B, T] or [S])."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.get_device() != dev:
        _refuse(name, t, dev, dtypes, shape)
    stride = t.stride()
    width = shape[-1]
    if stride[-1] != 1 and width > 1:
        raise ValueError(f"{name}: the elements of one token must be contiguous")
    if len(shape) == lead + 2:
        if stride[-2] != width and shape[-2] > 1:
            raise ValueError(f"{name}: the elements of one token must be contiguous")
        width *= shape[-2]
    if lead == 1:
        step = stride[0] if shape[0] > 1 else width
    elif shape[1] > 1:
        step = stride[1]
        if shape[0] > 1 and stride[0] != shape[1] * step:
            raise ValueError(f"{name}: batch rows must follow one another at the token stride")
    else:
        step = stride[0] if shape[0] > 1 else width
    return t.data_ptr(), step


def _dense(name, t, dev, dtypes, shape):
    """Check an optional contiguous tensor (a parameter or a state); returns its address or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or (shape is not None and t.shape != shape) or t.get_device() != dev:
        _refuse(name, t, dev, dtypes, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {tuple(ACTS)}, got {act!r}")
    return ACTS[act]


def _call(fn, dev, *args):
    """One library call on the current stream of device ``dev``."""
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _raise(status)


def _varlen(cu_seqlens, dev, B):
    """Address of the bounds, their N, and the number of sequences."""
    if cu_seqlens is None:
        return None, 0, B
    p = _dense("cu_seqlens", cu_seqlens, dev, (torch.int64,), None)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N+1] with N >= 1")
    return p, cu_seqlens.numel() - 1, cu_seqlens.numel() - 1


def _taps(weight, bias, dev, C):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    return _dense("weight", weight, dev, (_F32,), (C, W)), _dense("bias", bias, dev, (_F32,), (C,)), W


def conv(x, weight, out, bias=None, silu=True, initial_state=None, final_state=None, cu_seqlens=None):
    """Short causal convolution ``kda_conv``: ``x``, ``out`` bf16 [B, T, C] (token-strided views
    allowed), ``weight`` fp32 [C, W] (W = 2, 3, 4; the last tap is the token's own), ``bias`` fp32
    [C], states bf16 [B|N, W - 1, C] (the same buffer allowed). ``silu`` applies u sigmoid(u).
    Returns ``(out, final_state)``."""
    dev = _x_device(x, (3,), "[B, T, C]")
    shape = x.shape
    B, T, C = shape
    xp, xs = _rows("x", x, shape, 2, dev)
    op, os_ = _rows("out", out, shape, 2, dev)
    wp, bp, W = _taps(weight, bias, dev, C)
    cu, N, S = _varlen(cu_seqlens, dev, B)
    ip = _dense("initial_state", initial_state, dev, (_BF16,), (S, W - 1, C))
    fp = _dense("final_state", final_state, dev, (_BF16,), (S, W - 1, C))
    _call(_lib.kda_conv, dev, xp, xs, wp, bp, 2 if silu else 0, op, os_, ip, fp, cu, N, B, T, C, W)
    return out, final_state


def conv_step(x, weight, out, state, bias=None, silu=True):
    """``conv`` for one token of S sequences: ``x``, ``out`` bf16 [S, C] (``out`` may be ``x``),
    ``state`` bf16 [S, W - 1, C] updated in place. Returns ``(out, state)``."""
    dev = _x_device(x, (2,), "[S, C]")
    shape = x.shape
    S, C = shape
    xp, xs = _rows("x", x, shape, 1, dev)
    op, os_ = _rows("out", out, shape, 1, dev)
    wp, bp, W = _taps(weight, bias, dev, C)
    if state is None:
        raise ValueError("state is required")
    sp = _dense("state", state, dev, (_BF16,), (S, W - 1, C))
    _call(_lib.kda_conv_step, dev, xp, xs, wp, bp, 2 if silu else 0, op, os_, sp, S, C, W)
    return out, state


def _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, lead, dev):
    shape = x.shape
    tok, (H, P) = shape[:lead], shape[lead:]
    if not isinstance(b, torch.Tensor) or b.dim() != lead + 2:
        raise ValueError("b and c must be [..., G, 128]")
    gk = tok + b.shape[lead:]
    head = (*_rows("x", x, shape, lead, dev), *_rows("dt", dt, tok + (H,), lead, dev), *_rows("b", b, gk, lead, dev),
            *_rows("c", c, gk, lead, dev))
    if A_log is None:
        raise ValueError("A_log is required")
    params = tuple(_dense(name, t, dev, (_F32,), (H,)) for name, t in (("A_log", A_log), ("D", D), ("dt_bias", dt_bias)))
    return (*head, *params, *_rows("out", out, shape, lead, dev)), H, P, gk[lead], gk[lead + 1]


def ssm_workspace_bytes(states, tokens, H, P) -> int:
    """Bytes of workspace with which ``ssm`` may split the time axis of a call with ``states``
    sequences, ``tokens`` tokens in all and ``H`` heads of ``P`` channels on the current device
    (0: it would not split). Never more than 24 x SMs x (128 P + 1), so that one buffer of that
    size serves calls of any sizes."""
    n = _Z(0)
    _raise(_lib.kda_ssm_workspace_bytes(int(states), int(tokens), int(H), int(P), ctypes.byref(n)))
    return int(n.value)


def ssm(x, dt, b, c, out, A_log, D=None, dt_bias=None, initial_state=None, final_state=None, cu_seqlens=None,
        workspace=None):
    """Selective state-space scan ``kda_ssm``: ``x``, ``out`` bf16 [B, T, H, P] (P = 64 or 128),
    ``dt`` bf16 [B, T, H] before ``dt_bias`` and softplus, ``b``, ``c`` bf16 [B, T, G, 128] (G
    divides H), ``A_log``, ``D``, ``dt_bias`` fp32 [H], states bf16/fp32 [B|N, H, P, 128]. A CUDA
    uint8 ``workspace`` of ``ssm_workspace_bytes`` bytes lets calls with few (sequence, head) pairs
    split the time axis. Returns ``(out, final_state)``."""
    dev = _x_device(x, (4,), "[B, T, H, P]")
    B, T = x.shape[:2]
    head, H, P, G, K = _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, 2, dev)
    cu, N, S = _varlen(cu_seqlens, dev, B)
    ip = _dense("initial_state", initial_state, dev, (_BF16, _F32), (S, H, P, K))
    fp = _dense("final_state", final_state, dev, (_BF16, _F32), (S, H, P, K))
    wp = _dense("workspace", workspace, dev, (torch.uint8,), None)
    nbytes = workspace.numel() if wp else 0
    _call(_lib.kda_ssm, dev, *head, ip, DTYPE_NONE if ip is None else _CODES[initial_state.dtype],
          fp, DTYPE_NONE if fp is None else _CODES[final_state.dtype], cu, N, B, T, H, P, G, K, wp if nbytes else None, nbytes)
    return out, final_state


def ssm_step(x, dt, b, c, out, state, A_log, D=None, dt_bias=None):
    """``ssm`` for one token of S sequences: ``x``, ``out`` bf16 [S, H, P], ``dt`` bf16 [S, H],
    ``b``, ``c`` bf16 [S, G, 128], ``state`` bf16/fp32 [S, H, P, 128] updated in place. Returns
    ``(out, state)``."""
    dev = _x_device(x, (3,), "[S, H, P]")
    head, H, P, G, K = _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, 1, dev)
    S = x.shape[0]
    if state is None:
        raise ValueError("state is required")
    sp = _dense("state", state, dev, (_BF16, _F32), (S, H, P, K))
    _call(_lib.kda_ssm_step, dev, *head, sp, _CODES[state.dtype], S, H, P, G, K)
    return out, state


def gated_norm(x, gate, weight, out, act="sigmoid", gate_first=False, eps=1e-5):
    """RMS norm of a mixer's output rows with its output gate, ``kda_gated_norm``: ``x``, ``gate``,
    ``out`` bf16 [B, T, R, D] or [S, R, D], rows of D channels; ``weight`` fp32 [D], [R, D] or None.
    ``gate_first`` multiplies by ``act(gate)`` before the norm, else after it. ``out`` may be ``x``
    or ``gate``. Returns ``out``."""
    dev = _x_device(x, (3, 4), "[B, T, R, D] or [S, R, D]")
    shape = x.shape
    lead = len(shape) - 2
    R, D = shape[lead:]
    xp, xs = _rows("x", x, shape, lead, dev)
    zp, zs = _rows("gate", gate, shape, lead, dev)
    op, os_ = _rows("out", out, shape, lead, dev)
    per_row = isinstance(weight, torch.Tensor) and weight.dim() == 2
    wp = _dense("weight", weight, dev, (_F32,), (R, D) if per_row else (D,))
    M = shape[0] * shape[1] if lead == 2 else shape[0]
    _call(_lib.kda_gated_norm, dev, xp, xs, zp, zs, wp, R if per_row else 1, op, os_, eps, _act(act), int(bool(gate_first)), M, R, D)
    return out


def residual_norm(x, residual, residual_out, weight=None, out=None, post_weight=None, gate=None, act="none",
                  channel_scale=None, alpha=1.0, eps=1e-5):
    """Between two blocks, ``kda_residual_norm``: r' = residual + alpha channel_scale act(gate) n(x)
    and out = norm(r') weight in one pass. ``x``, ``gate``, ``out`` bf16 [B, T, D] or [S, D];
    ``residual``, ``residual_out`` bf16 or fp32 (the same buffer allowed; ``residual_out`` None: not
    written); ``weight``, ``post_weight``, ``channel_scale`` fp32 [D] or None. n(x) is x, or its RMS
    norm times ``post_weight`` where that is given. Returns ``(out, residual_out)``."""
    dev = _x_device(x, (2, 3), "[B, T, D] or [S, D]")
    shape = x.shape
    lead = len(shape) - 1
    D = shape[lead]
    xp, xs = _rows("x", x, shape, lead, dev)
    rp, rs = _rows("residual", residual, shape, lead, dev, (_BF16, _F32))
    rop, ros = (None, D) if residual_out is None else _rows("residual_out", residual_out, shape, lead, dev, (residual.dtype,))
    zp, zs = (None, D) if gate is None else _rows("gate", gate, shape, lead, dev)
    op, os_ = (None, D) if out is None else _rows("out", out, shape, lead, dev)
    pw, ch, w = (_dense(name, t, dev, (_F32,), (D,)) for name, t in
                 (("post_weight", post_weight), ("channel_scale", channel_scale), ("weight", weight)))
    M = shape[0] * shape[1] if lead == 2 else shape[0]
    _call(_lib.kda_residual_norm, dev, xp, xs, rp, rs, rop, ros, _CODES[residual.dtype], zp, zs, _act(act), pw, ch, alpha, w,
          op, os_, eps, M, D)
    return out, residual_out
