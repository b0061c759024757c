"""Rotary positions of queries and keys, and their norm for each head.

Thin binding over the C ABI of ``include/pamm_positions.h`` (the same
``libpamm.so``), in the manner of block_ops: PyTorch supplies device memory and
the stream, every step runs in the library's HIP kernels, there is no CPU
fallback, and all calls are asynchronous on the current stream or ``stream``.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check_workspace, _on_gpu, load_library
from .block_ops import _HEADS, _code, _heads_tensor, _launch, _not_overlapping, _pack_heads, _stream_of, _under, _vector, _ws

__all__ = ["rotary", "rotary_frequencies", "qk_norm_rotary", "qk_norm_rotary_backward",
           "qk_norm_rotary_backward_workspace_size"]

_sz, _vp = ctypes.c_size_t, ctypes.c_void_p

# pamm_rotary_t
_pack_rotary = struct.Struct("@4i6q2fPPqqPPP" + 4 * _HEADS).pack

_POSITION_EXPORTS = {
    "pamm_rotary": (ctypes.c_int, [_vp, _vp]),
    "pamm_rotary_backward_workspace_size": (_sz, [_vp]),
    "pamm_rotary_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}
_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = load_library()
        for name, (res, args) in _POSITION_EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _bound = lib
    return _bound


def rotary_frequencies(dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, turns=(1.0, 32.0), device="cuda"):
    """(inv_freq [dim / 2] float64 on ``device``, magnitude) for ``rotary``:
    radians a position of each pair, base^(-2 j / dim), and what cosines and
    sines are multiplied by.

    scaling, for contexts ``factor`` times as long as in training:
      "linear": every frequency divided by factor;
      "ntk":    a larger base, base * factor^(dim / (dim - 2)), which leaves the
                highest frequency and divides the lowest by factor;
      "yarn":   pairs that turn at least turns[1] times over original_length
                positions stay, those that turn at most turns[0] times are
                divided by factor, between the two a mix that is linear in
                j; magnitude 0.1 log(factor) + 1."""
    where = "rotary_frequencies"
    dim, base, factor = int(dim), float(base), float(factor)
    if dim < 0 or dim % 2:
        raise ValueError(f"{where}: dim must be even and not negative, got {dim}")
    if not base > 0.0 or not math.isfinite(base):
        raise ValueError(f"{where}: base must be positive, got {base}")
    if not factor >= 1.0 or not math.isfinite(factor):
        raise ValueError(f"{where}: factor must be at least 1, got {factor}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"{where}: scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if scaling is None and factor != 1.0:
        raise ValueError(f"{where}: a factor needs a scaling")
    if scaling == "ntk" and dim > 2:
        base *= factor ** (dim / (dim - 2))
    j = torch.arange(dim // 2, dtype=torch.float64)
    f, magnitude = base ** (-2.0 * j / max(dim, 1)), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        low, high = (float(t) for t in turns)
        if original_length is None or original_length < 1 or not 0.0 < low < high or base <= 1.0:
            raise ValueError(f"{where}: 'yarn' needs original_length, 0 < turns[0] < turns[1] and a base above 1")

        def pair(t):  # the (fractional) pair that turns t times over original_length positions
            return dim * math.log(original_length / (2.0 * math.pi * t)) / (2.0 * math.log(base))

        first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), dim - 1)
        mix = ((j - first) / max(last - first, 0.001)).clamp(0.0, 1.0)  # 0: stays, 1: divided
        f = f * (1.0 - mix) + f / factor * mix
        magnitude = 0.1 * math.log(factor) + 1.0
    return f.to(device), magnitude


def _positions(where, positions, offset, B, S):
    """(pointer, is int64, strides, offset's pointer)"""
    p = (0, 0, 0, 0)
    if positions is not None:
        if positions.dtype not in (torch.int64, torch.int32):
            raise TypeError(f"{where}: positions must be int64 or int32, got {positions.dtype}")
        if positions.shape == (S,):
            p = (positions.data_ptr(), int(positions.dtype == torch.int64), 0, positions.stride(0))
        elif positions.shape == (B, S):
            p = (positions.data_ptr(), int(positions.dtype == torch.int64), positions.stride(0), positions.stride(1))
        else:
            raise ValueError(f"{where}: positions must have shape {(S,)} or {(B, S)}, got {tuple(positions.shape)}")
    if offset is None:
        return (*p, 0)
    if offset.dim() != 1 or offset.shape[0] != B or not offset.is_contiguous():
        raise ValueError(f"{where}: offset must be contiguous of shape {(B,)}, got {tuple(offset.shape)}")
    if offset.dtype != torch.int32:
        raise TypeError(f"{where}: offset must be int32, got {offset.dtype}")
    return (*p, offset.data_ptr())


def _frequencies(where, inv_freq, D):
    if inv_freq is None:
        return 0, 0
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"{where}: inv_freq must be 1-D and contiguous, got shape {tuple(inv_freq.shape)}")
    if inv_freq.dtype != torch.float64:
        raise TypeError(f"{where}: inv_freq must be float64 (32 bits lose the angles of far positions), got "
                        f"{inv_freq.dtype}")
    if 2 * inv_freq.shape[0] > D:
        raise ValueError(f"{where}: {inv_freq.shape[0]} pairs do not fit a head dimension of {D}")
    return 2 * inv_freq.shape[0], inv_freq.data_ptr()


def _like(where, name, t, like):
    """``t``, or a tensor for results of ``like``'s shape, as (tensor, its packed layout)."""
    if t is None:
        t = torch.empty_like(like)
    else:
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError(f"{where}: {name} must be {like.dtype} of shape {tuple(like.shape)}, got "
                             f"{tuple(t.shape)} {t.dtype}")
        _not_overlapping(where, name, t)
    return t, _heads_tensor(where, name, t)


def _problem(where, q, k, qo, ko, q_weight, k_weight, inv_freq, positions, offset, interleaved, magnitude, eps, inverse,
             **others):
    """The GPU, and the checked arguments as a packed pamm_rotary_t; qo and ko are (tensor, layout)."""
    qh, (B, S, H, D) = _heads_tensor(where, "q" if k is not None else "x", q), q.shape
    kh = koh = (0, 0, 0, 0)
    Hk = 0
    if k is not None:
        kh, Hk = _heads_tensor(where, "k", k), k.shape[2]
        if (k.shape[0], k.shape[1], k.shape[3]) != (B, S, D) or Hk < 1:
            raise ValueError(f"{where}: k must be [{B} x {S} x heads x {D}], got {tuple(k.shape)}")
        if k.dtype != q.dtype:
            raise TypeError(f"{where}: q and k must share a dtype, got {q.dtype} and {k.dtype}")
        koh = ko[1]
    code = _code(where, q)
    wq = wk = 0
    if q_weight is not None:
        _vector(where, "q_weight", q_weight, D, q.dtype)
        _vector(where, "k_weight", k_weight, D, q.dtype)
        wq, wk = q_weight.data_ptr(), k_weight.data_ptr()
    rot, freq = _frequencies(where, inv_freq, D)
    *pos, off = _positions(where, positions, offset, B, S)
    index = q.get_device()
    for t in (q, k, q_weight, k_weight, inv_freq, positions, offset, *others.values()):
        if t is not None and (index < 0 or t.get_device() != index):
            _on_gpu(where, q=q, k=k, q_weight=q_weight, k_weight=k_weight, inv_freq=inv_freq, positions=positions,
                    offset=offset, **others)  # says which
    return index, _pack_rotary(code, int(bool(interleaved)), int(bool(inverse)), pos[1], B, S, H, Hk, D, rot,
                        float(magnitude), float(eps), freq, pos[0], pos[2], pos[3], off, wq, wk, *qh, *kh, *qo[1], *koh)


def rotary(x, inv_freq, *, positions=None, offset=None, interleaved: bool = False, magnitude: float = 1.0,
           inverse: bool = False, out=None, stream=None):
    """x [B x S x H x D] with the first 2 len(inv_freq) elements of each head row
    rotated by its token's position; the rest is copied.

    inv_freq: float64, radians a position of each pair (``rotary_frequencies``).
    Pair j is the elements j and j + len(inv_freq), with interleaved 2 j and
    2 j + 1.  The position of token s of sequence b is positions[b, s] (int64 or
    int32, [B x S] or [S]; s by default) + offset[b] ([B] int32, for instance a
    cache's lengths).  Angles are formed in 64 bits: cosines and sines are within
    4 * 2^-24 + |position * inv_freq| * 2^-51, which at 2^31 radians is another
    2^-20 (from 2^53 on positions themselves are rounded).  They are
    multiplied by magnitude.

    inverse turns by the negative angles: rotary(dy, ..., inverse=True) is the
    gradient of x and, with a magnitude of 1, takes x's rotation back.
    Queries and keys that lie side by side in a projection's packed output are
    one call.  out may be x itself, and must not share memory with it in any
    other way.  bf16 or fp32, D as for ``attention``; any strides of the outer
    dimensions."""
    where = "rotary"
    if stream is not None:
        return _under(stream, where, x, rotary, x, inv_freq, positions=positions, offset=offset, interleaved=interleaved,
                      magnitude=magnitude, inverse=inverse, out=out)
    _heads_tensor(where, "x", x)
    if inv_freq is None:
        raise ValueError(f"{where}: inv_freq is needed")
    o = _like(where, "out", out, x)
    index, p = _problem(where, x, None, o, None, None, None, inv_freq, positions, offset, interleaved, magnitude, 0.0, inverse,
                 out=o[0])
    _launch("pamm_rotary", index, _lib().pamm_rotary, p, _stream_of(index))
    return o[0]


def _weights(where, q_weight, k_weight):
    if q_weight is None or k_weight is None:
        raise ValueError(f"{where}: q_weight and k_weight are needed")


def qk_norm_rotary(q, k, q_weight, k_weight, inv_freq, *, positions=None, offset=None, interleaved: bool = False,
                   magnitude: float = 1.0, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Queries q [B x S x H x D] and keys k [B x S x Hkv x D], each head row x
    made x / sqrt(mean(x^2) + eps) * weight and then rotated as by ``rotary``, in
    one pass.  Returns (q_out, k_out).

    q_weight, k_weight [D] of q's dtype; inv_freq None: the norm alone.
    Results are rounded once.  q_out and k_out may be q and k themselves where
    no gradient is wanted: the backward pass starts from q and k."""
    where = "qk_norm_rotary"
    if stream is not None:
        return _under(stream, where, q, qk_norm_rotary, q, k, q_weight, k_weight, inv_freq, positions=positions,
                      offset=offset, interleaved=interleaved, magnitude=magnitude, eps=eps, q_out=q_out, k_out=k_out)
    _heads_tensor(where, "q", q)
    _heads_tensor(where, "k", k)
    _weights(where, q_weight, k_weight)
    qo, ko = _like(where, "q_out", q_out, q), _like(where, "k_out", k_out, k)
    index, p = _problem(where, q, k, qo, ko, q_weight, k_weight, inv_freq, positions, offset, interleaved, magnitude, eps,
                 False, q_out=qo[0], k_out=ko[0])
    _launch("pamm_rotary", index, _lib().pamm_rotary, p, _stream_of(index))
    return qo[0], ko[0]


def qk_norm_rotary_backward_workspace_size(q, k) -> int:
    """Bytes of workspace ``qk_norm_rotary_backward`` needs for tensors of these
    shapes (the most over both layouts and all numbers of rotated pairs)."""
    where = "qk_norm_rotary_backward_workspace_size"
    _heads_tensor(where, "q", q)
    kh = _heads_tensor(where, "k", k)
    B, S, H, D = q.shape
    pack = lambda inter, rot: _pack_rotary(_code(where, q), inter, 0, 0, B, S, H, k.shape[2], D, rot, 1.0, 0.0, 0, 0, 0, 0,
                                           0, 0, 0, *kh, *kh, *kh, *kh)
    return max(int(_lib().pamm_rotary_backward_workspace_size(pack(i, r))) for i in (0, 1) for r in range(0, D + 1, 2))


def qk_norm_rotary_backward(dq, dk, q, k, q_weight, k_weight, inv_freq, *, positions=None, offset=None,
                            interleaved: bool = False, magnitude: float = 1.0, eps: float = 1e-6, dq_out=None,
                            dk_out=None, workspace=None, stream=None):
    """Gradients of ``qk_norm_rotary`` from dq and dk, those of its results, and
    its inputs q and k; the other arguments as they were given to it.

    Returns (dq_out, dk_out, dq_weight [D] fp32, dk_weight [D] fp32).  dq_out
    and dk_out may be dq and dk themselves.  The weights' gradients are sums
    over all tokens and heads, padding among them.  Bitwise deterministic."""
    where = "qk_norm_rotary_backward"
    if stream is not None:
        return _under(stream, where, q, qk_norm_rotary_backward, dq, dk, q, k, q_weight, k_weight, inv_freq,
                      positions=positions, offset=offset, interleaved=interleaved, magnitude=magnitude, eps=eps,
                      dq_out=dq_out, dk_out=dk_out, workspace=workspace)
    _heads_tensor(where, "q", q)
    _heads_tensor(where, "k", k)
    _weights(where, q_weight, k_weight)
    grads = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k)):
        layout = _heads_tensor(where, name, t)
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError(f"{where}: {name} must be {like.dtype} of shape {tuple(like.shape)}, got {tuple(t.shape)} "
                             f"{t.dtype}")
        grads.append(_pack_heads(*layout))
    qo, ko = _like(where, "dq_out", dq_out, q), _like(where, "dk_out", dk_out, k)
    index, p = _problem(where, q, k, qo, ko, q_weight, k_weight, inv_freq, positions, offset, interleaved, magnitude, eps,
                 False, dq=dq, dk=dk, dq_out=qo[0], dk_out=ko[0], workspace=workspace)
    _check_workspace(where, workspace)
    dw = torch.empty((2, q.shape[3]), dtype=torch.float32, device=q.device)
    dwq, dwk = dw.unbind(0)
    lib = _lib()
    ws, nbytes = _ws(lib.pamm_rotary_backward_workspace_size(p), q.device, workspace, where)
    _launch("pamm_rotary_backward", index, lib.pamm_rotary_backward, p, *grads, dwq.data_ptr(), dwk.data_ptr(), ws,
            nbytes, _stream_of(index))
    return qo[0], ko[0], dwq, dwk
