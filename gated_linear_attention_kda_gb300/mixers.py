"""The mixers beside KDA: the gated delta rule, the norm and rotation of queries and keys, the paged
cache of keys and values and the attention of single tokens over it (``include/kda.h``, "Mixers
beside KDA"). Argument marshalling only, in the manner of the operators around the mixer
(``block.py``): every function writes the buffers it is given on the current CUDA stream, allocates
nothing and returns them."""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE_NONE, FLAG_QK_L2NORM, _lib, _P, _F, _I, _I64, _raise
from .block import _BF16, _CODES, _F32, _Z, _call, _dense, _refuse, _rows, _varlen

_U32 = ctypes.c_uint32
_HEAD = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _F, _P, _I64, _P, _P]
_lib.kda_gdn.argtypes = _HEAD + [_P, _I, _P, _I, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _U32, _P]
_lib.kda_gdn_step.argtypes = _HEAD + [_P, _I, _I64, _I64, _I64, _I64, _I64, _U32, _P]
_lib.kda_qk_rope.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I, _F, _P, _P, _I64, _I, _I64, _I64, _I64, _I64, _P]
_lib.kda_kv_append.argtypes = [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _I, _P, _I, _F, _P, _I64,
                               _I64, _I64, _I64, _I64, _P]
_lib.kda_attn_step.argtypes = [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _F, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _Z, _P]
_lib.kda_attn_step_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, ctypes.POINTER(_Z)]
for _f in ("kda_gdn", "kda_gdn_step", "kda_qk_rope", "kda_kv_append", "kda_attn_step", "kda_attn_step_workspace_bytes"):
    getattr(_lib, _f).restype = _I


def _device(name, t, dims, layout):
    """The device of the leading argument, whose shape the others are checked against."""
    if not isinstance(t, torch.Tensor) or t.dim() not in dims:
        raise ValueError(f"{name} must be {layout}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _need(name, t):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _gdn_args(q, k, v, a, beta, scale, out, A_log, dt_bias, lead, dev):
    shape = v.shape
    tok, (H, V) = shape[:lead], shape[lead:]
    if not isinstance(q, torch.Tensor) or q.dim() != lead + 2:
        raise ValueError("q and k must be [..., HK, 128]")
    gk = tok + q.shape[lead:]
    head = (*_rows("q", q, gk, lead, dev), *_rows("k", k, gk, lead, dev), *_rows("v", v, shape, lead, dev),
            *_rows("a", a, tok + (H,), lead, dev), *_rows("beta", beta, tok + (H,), lead, dev), scale, *_rows("out", out, shape, lead, dev))
    params = (_dense("A_log", _need("A_log", A_log), dev, (_F32,), (H,)), _dense("dt_bias", dt_bias, dev, (_F32,), (H,)))
    return (*head, *params), H, gk[lead], gk[lead + 1], V


def gdn(q, k, v, a, beta, scale, out, A_log, dt_bias=None, initial_state=None, final_state=None, cu_seqlens=None, qk_l2norm=False):
    """Gated delta rule ``kda_gdn``: ``q``, ``k`` bf16 [B, T, HK, 128], ``v``, ``out`` bf16 [B, T, H, 128]
    (HK divides H; token-strided views allowed), ``a`` (before ``dt_bias`` and softplus) and ``beta``
    (before the sigmoid) bf16 [B, T, H], ``A_log``, ``dt_bias`` fp32 [H], states bf16/fp32
    [B|N, H, 128, 128]. ``qk_l2norm`` normalises q and k per (token, head). Sequences of up to 8 tokens
    run in fp32, longer ones in chunks with bf16 operands. Returns ``(out, final_state)``."""
    dev = _device("v", v, (4,), "[B, T, H, 128]")
    B, T = v.shape[:2]
    head, H, HK, K, V = _gdn_args(q, k, v, a, beta, scale, out, A_log, dt_bias, 2, dev)
    cu, N, S = _varlen(cu_seqlens, dev, B)
    ip = _dense("initial_state", initial_state, dev, (_BF16, _F32), (S, H, V, K))
    fp = _dense("final_state", final_state, dev, (_BF16, _F32), (S, H, V, K))
    _call(_lib.kda_gdn, dev, *head, ip, DTYPE_NONE if ip is None else _CODES[initial_state.dtype],
          fp, DTYPE_NONE if fp is None else _CODES[final_state.dtype], cu, N, B, T, H, HK, K, V, FLAG_QK_L2NORM if qk_l2norm else 0)
    return out, final_state


def gdn_step(q, k, v, a, beta, scale, out, state, A_log, dt_bias=None, qk_l2norm=False):
    """``gdn`` for one token of S sequences: ``q``, ``k`` bf16 [S, HK, 128], ``v``, ``out`` bf16 [S, H, 128],
    ``a``, ``beta`` bf16 [S, H], ``state`` bf16/fp32 [S, H, 128, 128] updated in place. Returns ``(out, state)``."""
    dev = _device("v", v, (3,), "[S, H, 128]")
    head, H, HK, K, V = _gdn_args(q, k, v, a, beta, scale, out, A_log, dt_bias, 1, dev)
    S = v.shape[0]
    sp = _dense("state", _need("state", state), dev, (_BF16, _F32), (S, H, V, K))
    _call(_lib.kda_gdn_step, dev, *head, sp, _CODES[state.dtype], S, H, HK, K, V, FLAG_QK_L2NORM if qk_l2norm else 0)
    return out, state


def _turn(inv_freq, dev):
    p = _dense("inv_freq", inv_freq, dev, (_F32,), None)
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [R / 2]")
    return p, 0 if inv_freq is None else 2 * inv_freq.numel()


def qk_rope(q, k, q_out, k_out, positions, inv_freq=None, q_weight=None, k_weight=None, norm=True, interleaved=False, eps=1e-6):
    """Heads of queries and keys normed and turned in one pass, ``kda_qk_rope``: ``q``, ``q_out`` bf16
    [B, T, H, D] or [S, H, D] (D = 64, 128, 256), ``k``, ``k_out`` the same with HK heads, or both None;
    ``positions`` int64 [B, T] or [S]; ``inv_freq`` fp32 [R / 2] (the first R channels are turned, R a multiple
    of 16; None: none are), weights fp32 [D] or None. Pairs are (i, i + R / 2), or neighbours if ``interleaved``.
    ``q_out`` may be ``q`` and ``k_out`` ``k``. Returns ``(q_out, k_out)``."""
    dev = _device("q", q, (3, 4), "[B, T, H, D] or [S, H, D]")
    shape = q.shape
    lead = len(shape) - 2
    tok, (H, D) = shape[:lead], shape[lead:]
    qp, qs = _rows("q", q, shape, lead, dev)
    qop, qos = _rows("q_out", q_out, shape, lead, dev)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out come together")
    kp, ks, kop, kos, HK = None, 0, None, 0, 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != lead + 2:
            raise ValueError("k must have q's layout")
        HK = k.shape[lead]
        kshape = tok + (HK, D)
        kp, ks = _rows("k", k, kshape, lead, dev)
        kop, kos = _rows("k_out", k_out, kshape, lead, dev)
    pp = _dense("positions", _need("positions", positions), dev, (torch.int64,), tok)
    fp, R = _turn(inv_freq, dev)
    qw, kw = (_dense(n, w, dev, (_F32,), (D,)) for n, w in (("q_weight", q_weight), ("k_weight", k_weight)))
    M = shape[0] * shape[1] if lead == 2 else shape[0]
    _call(_lib.kda_qk_rope, dev, qp, qs, kp, ks, qop, qos, kop, kos, qw, kw, int(bool(norm)), eps, pp, fp, R, int(bool(interleaved)),
          M, H, HK, D)
    return q_out, k_out


def _pages(k_cache, v_cache, page_table, S, HK, D, dev):
    """Check the caches and the table; returns their addresses and sizes in the order of the library's calls."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, HK, page_size, D]")
    shape = (k_cache.shape[0], HK, k_cache.shape[2], D)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.dtype != _BF16 or t.shape != shape or t.get_device() != dev:
            _refuse(name, t, dev, (_BF16,), shape)
        if t.stride()[1:] != (shape[2] * D, D, 1):
            raise ValueError(f"{name}: the elements of one page must be contiguous")
        if shape[0] > 1 and t.stride(0) != k_cache.stride(0):
            raise ValueError("k_cache and v_cache must have the same page stride")
    stride = k_cache.stride(0) if shape[0] > 1 else HK * shape[2] * D
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [S, pages per sequence]")
    tp = _dense("page_table", page_table, dev, (torch.int32,), (S, page_table.shape[1]))
    return k_cache.data_ptr(), v_cache.data_ptr(), stride, shape[0], shape[2], tp, page_table.shape[1]


def kv_append(k, v, k_cache, v_cache, page_table, positions, inv_freq=None, k_weight=None, norm=False, interleaved=False, eps=1e-6,
              cu_seqlens=None):
    """Keys and values of new tokens into a paged cache, ``kda_kv_append``: ``k``, ``v`` bf16 [B, T, HK, D] or
    [S, HK, D] (one token per sequence), caches bf16 [pages, HK, page_size, D] (views with a page stride
    allowed), ``page_table`` int32 [B|N|S, pages per sequence], ``positions`` int64 [B, T] or [S] (below 0: the
    token is not written). Keys are normed and turned as in ``qk_rope``. Returns ``(k_cache, v_cache)``."""
    dev = _device("k", k, (3, 4), "[B, T, HK, D] or [S, HK, D]")
    shape = k.shape
    lead = len(shape) - 2
    tok, (HK, D) = shape[:lead], shape[lead:]
    kp, ks = _rows("k", k, shape, lead, dev)
    vp, vs = _rows("v", v, shape, lead, dev)
    B, T = tok if lead == 2 else (tok[0], 1)
    if cu_seqlens is not None and lead == 1:
        raise ValueError("cu_seqlens needs k as [1, T, HK, D]")
    cu, N, S = _varlen(cu_seqlens, dev, B)
    pages = _pages(k_cache, v_cache, page_table, S, HK, D, dev)
    pp = _dense("positions", _need("positions", positions), dev, (torch.int64,), tok)
    fp, R = _turn(inv_freq, dev)
    kw = _dense("k_weight", k_weight, dev, (_F32,), (D,))
    _call(_lib.kda_kv_append, dev, kp, ks, vp, vs, *pages, pp, fp, R, int(bool(interleaved)), kw, int(bool(norm)), eps, cu, N, B, T, HK, D)
    return k_cache, v_cache


def attn_step_workspace_bytes(S, H, HK, D) -> int:
    """Bytes of workspace with which ``attn_step`` may cut the caches of ``S`` sequences on the current device,
    whatever their lengths."""
    n = _Z(0)
    _raise(_lib.kda_attn_step_workspace_bytes(int(S), int(H), int(HK), int(D), ctypes.byref(n)))
    return int(n.value)


def attn_step(q, k_cache, v_cache, page_table, positions, out, scale, lse=None, workspace=None):
    """Softmax attention of one new token per sequence over a paged cache, ``kda_attn_step``: ``q``, ``out`` bf16
    [S, H, D] (D = 64, 128; the caches' HK heads divide H), caches and ``page_table`` as in ``kv_append``,
    ``positions`` int64 [S] of the new tokens, which see the cache up to themselves (below 0: out is 0), ``lse``
    fp32 [S, H]. Give a CUDA uint8 ``workspace`` of ``attn_step_workspace_bytes`` bytes: without it one warp reads all of a
    sequence's keys and values of a key head, 10 to 80 times slower for one long sequence. Returns ``(out, lse)``."""
    dev = _device("q", q, (3,), "[S, H, D]")
    shape = q.shape
    S, H, D = shape
    qp, qs = _rows("q", q, shape, 1, dev)
    op, os_ = _rows("out", out, shape, 1, dev)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, HK, page_size, D]")
    HK = k_cache.shape[1]
    pages = _pages(k_cache, v_cache, page_table, S, HK, D, dev)
    pp = _dense("positions", _need("positions", positions), dev, (torch.int64,), (S,))
    lp = _dense("lse", lse, dev, (_F32,), (S, H))
    wp = _dense("workspace", workspace, dev, (torch.uint8,), None)
    nbytes = workspace.numel() if wp else 0
    _call(_lib.kda_attn_step, dev, qp, qs, *pages, pp, scale, op, os_, lp, S, H, HK, D, wp if nbytes else None, nbytes)
    return out, lse
