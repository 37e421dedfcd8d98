"""The operators around the mixer: short causal convolution, selective state-space scan, gated norm
and residual norm, for prompts and for single tokens (``include/kda.h``, "Operators around the
mixer"). Argument marshalling only, as in the package's other calls: every function writes the
buffers it is given on the current CUDA stream, allocates nothing and returns them.

Token axes may be strided: a slice of a projection's row is passed as it stands. The elements of
one token are contiguous, and batch rows follow one another at the token stride.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _lib, _P, _F, _I, _I64, _ptr, _raise, _same_device, _state_code

_Z = ctypes.c_size_t
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


def _rows(name, t, shape, lead, dtype=torch.bfloat16):
    """Check an activation of the given shape and return the distance in elements between its
    tokens; the first ``lead`` dimensions are the token axes ([B, T] or [S])."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    width = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] > 1 and t.stride(i) != width:
            raise ValueError(f"{name}: the elements of one token must be contiguous")
        width *= t.shape[i]
    axes = [i for i in range(lead) if t.shape[i] > 1]
    if not axes or t.numel() == 0:
        return width
    stride = t.stride(axes[-1])
    if len(axes) == 2 and t.stride(axes[0]) != t.shape[axes[1]] * stride:
        raise ValueError(f"{name}: batch rows must follow one another at the token stride")
    return stride


def _param(name, t, shape):
    _check(name, t, torch.float32, shape, True)


def _act(act, allowed=("none", "sigmoid", "silu")):
    if act not in allowed:
        raise ValueError(f"act must be one of {allowed}, got {act!r}")
    return ACTS[act]


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _varlen(cu_seqlens, B):
    if cu_seqlens is None:
        return 0, B
    _check("cu_seqlens", cu_seqlens, torch.int64, None, True)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N+1] with N >= 1")
    return cu_seqlens.numel() - 1, cu_seqlens.numel() - 1


def conv(x, weight, out, bias=None, silu=True, initial_state=None, final_state=None, cu_seqlens=None):
    """Short causal convolution ``kda_conv``: ``x``, ``out`` bf16 [B, T, C] (token-strided views
    allowed), ``weight`` fp32 [C, W] (W = 2, 3, 4; the last tap is the token's own), ``bias`` fp32
    [C], states bf16 [B|N, W - 1, C] (the same buffer allowed). ``silu`` applies u sigmoid(u).
    Returns ``(out, final_state)``."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    xs, os_ = _rows("x", x, x.shape, 2), _rows("out", out, x.shape, 2)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    _param("weight", weight, (C, W))
    _param("bias", bias, (C,))
    N, S = _varlen(cu_seqlens, B)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        _check(name, t, torch.bfloat16, (S, W - 1, C), True)
    _same_device(x.device, (("weight", weight), ("out", out), ("bias", bias), ("initial_state", initial_state),
                            ("final_state", final_state), ("cu_seqlens", cu_seqlens)))
    with torch.cuda.device(x.device):
        _raise(_lib.kda_conv(_ptr(x), xs, _ptr(weight), _ptr(bias), ACTS["silu" if silu else "none"], _ptr(out), os_,
                             _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens), N, B, T, C, W, _stream(x.device)))
    return out, final_state


def conv_step(x, weight, out, state, bias=None, silu=True):
    """``conv`` for one token of S sequences: ``x``, ``out`` bf16 [S, C] (``out`` may be ``x``),
    ``state`` bf16 [S, W - 1, C] updated in place. Returns ``(out, state)``."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [S, C]")
    S, C = x.shape
    xs, os_ = _rows("x", x, x.shape, 1), _rows("out", out, x.shape, 1)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    _param("weight", weight, (C, W))
    _param("bias", bias, (C,))
    if state is None:
        raise ValueError("state is required")
    _check("state", state, torch.bfloat16, (S, W - 1, C), True)
    _same_device(x.device, (("weight", weight), ("out", out), ("bias", bias), ("state", state)))
    with torch.cuda.device(x.device):
        _raise(_lib.kda_conv_step(_ptr(x), xs, _ptr(weight), _ptr(bias), ACTS["silu" if silu else "none"], _ptr(out), os_,
                                  _ptr(state), S, C, W, _stream(x.device)))
    return out, state


def _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, lead):
    tok, (H, P) = tuple(x.shape[:lead]), x.shape[lead:]
    if not isinstance(b, torch.Tensor) or b.dim() != lead + 2:
        raise ValueError("b and c must be [..., G, 128]")
    G, K = b.shape[lead:]
    strides = [_rows("x", x, x.shape, lead), _rows("dt", dt, tok + (H,), lead), _rows("b", b, tok + (G, K), lead),
               _rows("c", c, tok + (G, K), lead), _rows("out", out, x.shape, lead)]
    if A_log is None:
        raise ValueError("A_log is required")
    for name, t in (("A_log", A_log), ("D", D), ("dt_bias", dt_bias)):
        _param(name, t, (H,))
    _same_device(x.device, (("dt", dt), ("b", b), ("c", c), ("out", out), ("A_log", A_log), ("D", D), ("dt_bias", dt_bias)))
    head = (_ptr(x), strides[0], _ptr(dt), strides[1], _ptr(b), strides[2], _ptr(c), strides[3], _ptr(A_log), _ptr(D),
            _ptr(dt_bias), _ptr(out), strides[4])
    return head, H, P, G, K


def ssm_workspace_bytes(states, tokens, H, P) -> int:
    """Bytes of workspace with which ``ssm`` may split the time axis of a call with ``states``
    sequences, ``tokens`` tokens in all and ``H`` heads of ``P`` channels on the current device
    (0: it would not split)."""
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
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be [B, T, H, P]")
    B, T = x.shape[:2]
    head, H, P, G, K = _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, 2)
    N, S = _varlen(cu_seqlens, B)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        _check(name, t, None, (S, H, P, K), True)
    nbytes = 0
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        nbytes = workspace.numel()
    _same_device(x.device, (("initial_state", initial_state), ("final_state", final_state), ("cu_seqlens", cu_seqlens),
                            ("workspace", workspace)))
    with torch.cuda.device(x.device):
        _raise(_lib.kda_ssm(*head, _ptr(initial_state), _state_code(initial_state), _ptr(final_state),
                            _state_code(final_state), _ptr(cu_seqlens), N, B, T, H, P, G, K,
                            _ptr(workspace) if nbytes else None, nbytes, _stream(x.device)))
    return out, final_state


def ssm_step(x, dt, b, c, out, state, A_log, D=None, dt_bias=None):
    """``ssm`` for one token of S sequences: ``x``, ``out`` bf16 [S, H, P], ``dt`` bf16 [S, H],
    ``b``, ``c`` bf16 [S, G, 128], ``state`` bf16/fp32 [S, H, P, 128] updated in place. Returns
    ``(out, state)``."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be [S, H, P]")
    head, H, P, G, K = _ssm_args(x, dt, b, c, out, A_log, D, dt_bias, 1)
    S = x.shape[0]
    if state is None:
        raise ValueError("state is required")
    _check("state", state, None, (S, H, P, K), True)
    _same_device(x.device, (("state", state),))
    with torch.cuda.device(x.device):
        _raise(_lib.kda_ssm_step(*head, _ptr(state), _state_code(state), S, H, P, G, K, _stream(x.device)))
    return out, state


def gated_norm(x, gate, weight, out, act="sigmoid", gate_first=False, eps=1e-5):
    """RMS norm of a mixer's output rows with its output gate, ``kda_gated_norm``: ``x``, ``gate``,
    ``out`` bf16 [B, T, R, D] or [S, R, D], rows of D channels; ``weight`` fp32 [D], [R, D] or None.
    ``gate_first`` multiplies by ``act(gate)`` before the norm, else after it. ``out`` may be ``x``
    or ``gate``. Returns ``out``."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("x must be [B, T, R, D] or [S, R, D]")
    lead = x.dim() - 2
    R, D = x.shape[lead:]
    xs, zs, os_ = (_rows(n, t, x.shape, lead) for n, t in (("x", x), ("gate", gate), ("out", out)))
    w_rows = 1
    if weight is not None:
        w_rows = R if isinstance(weight, torch.Tensor) and weight.dim() == 2 else 1
        _param("weight", weight, (R, D) if w_rows == R and weight.dim() == 2 else (D,))
    _same_device(x.device, (("gate", gate), ("weight", weight), ("out", out)))
    M = x.numel() // (R * D) if R * D else 0
    with torch.cuda.device(x.device):
        _raise(_lib.kda_gated_norm(_ptr(x), xs, _ptr(gate), zs, _ptr(weight), w_rows, _ptr(out), os_, float(eps), _act(act),
                                   int(bool(gate_first)), M, R, D, _stream(x.device)))
    return out


def residual_norm(x, residual, residual_out, weight=None, out=None, post_weight=None, gate=None, act="none",
                  channel_scale=None, alpha=1.0, eps=1e-5):
    """Between two blocks, ``kda_residual_norm``: r' = residual + alpha channel_scale act(gate) n(x)
    and out = norm(r') weight in one pass. ``x``, ``gate``, ``out`` bf16 [B, T, D] or [S, D];
    ``residual``, ``residual_out`` bf16 or fp32 (the same buffer allowed; ``residual_out`` None: not
    written); ``weight``, ``post_weight``, ``channel_scale`` fp32 [D] or None. n(x) is x, or its RMS
    norm times ``post_weight`` where that is given. Returns ``(out, residual_out)``."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be [B, T, D] or [S, D]")
    lead, D = x.dim() - 1, x.shape[-1]
    if not isinstance(residual, torch.Tensor):
        raise TypeError("residual must be a torch.Tensor")
    if residual.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"residual must be bfloat16 or float32, got {residual.dtype}")
    st = {"x": _rows("x", x, x.shape, lead), "residual": _rows("residual", residual, x.shape, lead, residual.dtype)}
    for name, t, dt in (("residual_out", residual_out, residual.dtype), ("gate", gate, torch.bfloat16), ("out", out, torch.bfloat16)):
        st[name] = D if t is None else _rows(name, t, x.shape, lead, dt)
    for name, t in (("post_weight", post_weight), ("channel_scale", channel_scale), ("weight", weight)):
        _param(name, t, (D,))
    _same_device(x.device, (("residual", residual), ("residual_out", residual_out), ("gate", gate), ("out", out),
                            ("post_weight", post_weight), ("channel_scale", channel_scale), ("weight", weight)))
    M = x.numel() // D if D else 0
    with torch.cuda.device(x.device):
        _raise(_lib.kda_residual_norm(_ptr(x), st["x"], _ptr(residual), st["residual"], _ptr(residual_out), st["residual_out"],
                                      _state_code(residual), _ptr(gate), st["gate"], _act(act), _ptr(post_weight),
                                      _ptr(channel_scale), float(alpha), _ptr(weight), _ptr(out), st["out"], float(eps), M, D,
                                      _stream(x.device)))
    return out, residual_out
