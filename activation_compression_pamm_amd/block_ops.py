"""The operators around a PAMM projection in a transformer block.

Thin binding over the C ABI of ``include/pamm_block.h`` (the same
``libpamm.so``): attention with a backward pass that recomputes its
probabilities, the residual addition with its root-mean-square norm (with an
output in 8 bits, and its backward pass), and the global gradient norm with
clipping.  "QKV Projections Require a Fraction of Their Memory", section 3
"Contributi Chiave", states that the method composes with attention that keeps
no probabilities; these are that attention and its neighbours.

As in the rest of the package, PyTorch supplies device memory and the stream,
every step runs in the library's HIP kernels, and there is no CPU fallback.
All calls are asynchronous on the current stream.  With ``stream`` they run as
under ``torch.cuda.stream(stream)``: what they allocate belongs to that stream,
so that no memory of work pending on another is written.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import BF16, F32, PammError, _check, _check_workspace, _empty_rows, _on_gpu, _ptr, load_library

__all__ = ["attention", "attention_backward", "attention_workspace_size", "attention_backward_workspace_size",
           "add_rms_norm", "add_rms_norm_fp8", "add_rms_norm_backward", "clip_grad_norm", "MAX_HEAD_DIM"]

MAX_HEAD_DIM = 128
_FLT_MAX = 3.4028234663852886e38

_i32, _i64, _f32, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class _Heads(ctypes.Structure):
    """pamm_heads_t"""
    _fields_ = [("data", _vp), ("stride_b", _i64), ("stride_s", _i64), ("stride_h", _i64)]


class _Attention(ctypes.Structure):
    """pamm_attention_t"""
    _fields_ = [("dtype", _i32), ("causal", _i32), ("batch", _i64), ("seq_q", _i64), ("seq_k", _i64),
                ("heads", _i64), ("heads_kv", _i64), ("head_dim", _i64), ("window", _i64), ("scale", _f32),
                ("q_len", _vp), ("kv_len", _vp), ("q", _Heads), ("k", _Heads), ("v", _Heads), ("o", _Heads),
                ("lse", _vp)]


class _Grad(ctypes.Structure):
    """pamm_grad_t"""
    _fields_ = [("data", _vp), ("out", _vp), ("rows", _i64), ("cols", _i64), ("ld", _i64), ("ld_out", _i64),
                ("dtype", _i32), ("out_dtype", _i32)]


# The same layouts for struct.pack, which builds one in a fraction of the time
# of a ctypes structure: these calls are as short as single tokens.
_HEADS = "Pqqq"
_pack_attention = struct.Struct("@ii7qf4xPP" + 4 * _HEADS + "P").pack
_pack_heads = struct.Struct("@" + _HEADS).pack
_pack_grad = struct.Struct("@PP4qii").pack

_BLOCK_EXPORTS = {
    "pamm_attention_workspace_size": (_sz, [_vp]),
    "pamm_attention": (ctypes.c_int, [_vp, _vp, _sz, _vp]),
    "pamm_attention_backward_workspace_size": (_sz, [_vp]),
    "pamm_attention_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pamm_add_rms_norm": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, ctypes.c_int, _f32, _vp, _i64, _vp,
                                         _i64, _vp, _i64, _vp, _vp, _vp]),
    "pamm_add_rms_norm_backward_workspace_size": (_sz, [_i64, _i64, ctypes.c_int]),
    "pamm_add_rms_norm_backward": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64,
                                                  ctypes.c_int, _vp, _i64, _vp, _vp, _sz, _vp]),
    "pamm_clip_grad_norm_workspace_size": (_sz, [_vp, _i64]),
    "pamm_clip_grad_norm": (ctypes.c_int, [_vp, _i64, _f32, _f32, _vp, _vp, _sz, _vp]),
}
_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = load_library()
        for name, (res, args) in _BLOCK_EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _bound = lib
    return _bound


_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _code(where, t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{where}: float32 and bfloat16 tensors are supported, got {t.dtype}")
    return code


def _ws(nbytes, device, workspace, where):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"{where}: workspace needs {nbytes} bytes")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _under(stream, where, t, call, *args, **kw):
    """call(*args) with ``stream``, which is on t's GPU, as the current one."""
    if t.is_cuda and stream.device != t.device:
        raise ValueError(f"{where}: stream is on {stream.device}, tensors are on {t.device}")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _stream_of(index):
    """The handle of torch's current stream on that GPU."""
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _launch(where, index, fn, *args):
    """fn(*args) with the tensors' GPU as the current one: kernels are launched
    on the device that their memory and stream belong to."""
    now = torch.cuda.current_device()
    if now == index:
        status = fn(*args)
    else:
        torch.cuda.set_device(index)
        try:
            status = fn(*args)
        finally:
            torch.cuda.set_device(now)
    if status != 0:
        _check(status, where)


# ------------------------------------------------------------------- attention

def _heads_tensor(where, name, t):
    if t.dim() != 4:
        raise ValueError(f"{where}: {name} must be 4-D [batch x sequence x heads x head_dim], "
                         f"got shape {tuple(t.shape)}")
    stride = t.stride()
    if stride[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{where}: {name} must have contiguous head rows (stride 1 in the last dimension)")
    return t.data_ptr(), stride[0], stride[1], stride[2]


def _lengths(where, name, t, batch):
    if t is None:
        return 0
    if t.dim() != 1 or t.shape[0] != batch:
        raise ValueError(f"{where}: {name} must have shape {(batch,)}, got {tuple(t.shape)}")
    if t.dtype != torch.int32:
        raise TypeError(f"{where}: {name} must be int32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    return t.data_ptr()


def _problem(where, q, k, v, o, lse, causal, window, scale, q_len, kv_len, **others):
    """The checked arguments as a packed pamm_attention_t."""
    qh, kh, vh = _heads_tensor(where, "q", q), _heads_tensor(where, "k", k), _heads_tensor(where, "v", v)
    oh = _heads_tensor(where, "o", o) if o is not None else (0, 0, 0, 0)
    dtype = q.dtype
    if k.dtype != dtype or v.dtype != dtype or (o is not None and o.dtype != dtype):
        raise TypeError(f"{where}: q, k, v and o must share a dtype, got {dtype}, {k.dtype}, {v.dtype}"
                        + (f" and {o.dtype}" if o is not None else ""))
    B, Sq, H, D = q.shape
    kshape = k.shape
    Bk, Sk, Hkv, Dk = kshape
    if Bk != B or Dk != D or v.shape != kshape:
        raise ValueError(f"{where}: k and v must be [{B} x sequence x heads x {D}], got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{where}: {H} query heads do not share {Hkv} key/value heads evenly")
    _on_gpu(where, q=q, k=k, v=v, o=o, lse=lse, q_len=q_len, kv_len=kv_len, **others)
    if o is not None and o.shape != q.shape:
        raise ValueError(f"{where}: o must have shape {(B, Sq, H, D)}, got {tuple(o.shape)}")
    if lse is not None and (lse.shape != (B, H, Sq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError(f"{where}: lse must be contiguous float32 of shape {(B, H, Sq)}")
    return _pack_attention(
        _code(where, q), 1 if causal else 0, B, Sq, Sk, H, Hkv, D, int(window or 0),
        1.0 / math.sqrt(max(D, 1)) if scale is None else float(scale), _lengths(where, "q_len", q_len, B),
        _lengths(where, "kv_len", kv_len, B), *qh, *kh, *vh, *oh, lse.data_ptr() if lse is not None else 0)


def attention_workspace_size(q, k, *, causal=False, kv_len=None) -> int:
    """Bytes of workspace ``attention`` needs for tensors of these shapes
    (more where the keys' lengths are given: they are cut finer)."""
    p = _problem("attention_workspace_size", q, k, k, None, None, causal, 0, None, None, kv_len)
    return int(_lib().pamm_attention_workspace_size(p))


def attention_backward_workspace_size(q, k, *, causal=False) -> int:
    """Bytes of workspace ``attention_backward`` needs for tensors of these shapes."""
    p = _problem("attention_backward_workspace_size", q, k, k, None, None, causal, 0, None, None, None)
    return int(_lib().pamm_attention_backward_workspace_size(p))


def _not_overlapping(where, name, t):
    """A written tensor must give every element an address of its own."""
    if t.is_contiguous():
        return
    need = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < need:
            raise ValueError(f"{where}: {name} is written and must not overlap itself, got strides {t.stride()} "
                             f"for shape {tuple(t.shape)}")
        need = stride * (size - 1) + need


def attention(q, k, v, *, causal: bool = False, window: int = 0, scale=None, q_len=None, kv_len=None, o=None,
              lse=None, workspace=None, stream=None):
    """softmax(scale q k^T) v for q [B x Sq x H x D], k and v [B x Sk x Hkv x D].

    H is a multiple of Hkv: query head h uses key/value head h // (H / Hkv).
    The outer dimensions may lie in any order (views of a packed projection
    output, transposed caches); D <= 128, a multiple of 8 (bf16) or 4 (fp32).
    scale defaults to 1 / sqrt(D).  q_len and kv_len [B] int32 give each
    sequence's valid rows (all by default); K and V past them are never read.
    With causal, query i sees the keys up to i + kv_len - q_len, so new tokens
    against a cache and padded training batches both line up; window > 0
    leaves only the last `window` of those.

    One query per sequence (or few) splits the keys over the whole device.
    Returns (o [B x Sq x H x D], lse [B x H x Sq] fp32); a query that sees no
    key has o = 0 and lse = -inf.  attention_backward takes both.  o and lse,
    where given, must not share memory with the inputs."""
    where = "attention"
    if stream is not None:
        return _under(stream, where, q, attention, q, k, v, causal=causal, window=window, scale=scale, q_len=q_len,
                      kv_len=kv_len, o=o, lse=lse, workspace=workspace)
    if q.dim() != 4:
        _heads_tensor(where, "q", q)
    if o is None:
        o = torch.empty_like(q) if q.stride(3) == 1 else None
    else:
        _heads_tensor(where, "o", o)
        _not_overlapping(where, "o", o)
    if lse is None:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
    p = _problem(where, q, k, v, o, lse, causal, window, scale, q_len, kv_len, workspace=workspace)
    _check_workspace(where, workspace)
    lib, index = _lib(), q.get_device()
    ws, nbytes = _ws(lib.pamm_attention_workspace_size(p), q.device, workspace, where)
    _launch("pamm_attention", index, lib.pamm_attention, p, ws, nbytes, _stream_of(index))
    return o, lse


def attention_backward(do, q, k, v, o, lse, *, causal: bool = False, window: int = 0, scale=None, q_len=None,
                       kv_len=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of ``attention`` from do, the gradient of its o,
    and its outputs; the other arguments as they were given to it.

    The probabilities are recomputed from q, k and lse, so nothing of size
    Sq x Sk exists.  dk and dv are summed over the query heads that share
    them.  dq, dk and dv may be given (strided views, for instance of one
    packed gradient); they are written whole, with zeros past the lengths, and
    must not share memory with each other or the inputs.
    Bitwise deterministic."""
    where = "attention_backward"
    if stream is not None:
        return _under(stream, where, q, attention_backward, do, q, k, v, o, lse, causal=causal, window=window,
                      scale=scale, q_len=q_len, kv_len=kv_len, dq=dq, dk=dk, dv=dv, workspace=workspace)
    doh = _heads_tensor(where, "do", do)
    if do.shape != q.shape or do.dtype != q.dtype:
        raise ValueError(f"{where}: do must be {q.dtype} of shape {tuple(q.shape)}, got {tuple(do.shape)} {do.dtype}")
    outs, packed = [], [_pack_heads(*doh)]
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            # like's own order if it is dense, else contiguous
            t = torch.empty_like(like)
            if t.stride(3) != 1 and t.shape[3] > 1:
                _heads_tensor(where, name[1:], like)
            _not_overlapping(where, name, t)
        else:
            _heads_tensor(where, name, t)
            if t.shape != like.shape or t.dtype != like.dtype:
                raise ValueError(f"{where}: {name} must be {like.dtype} of shape {tuple(like.shape)}, "
                                 f"got {tuple(t.shape)} {t.dtype}")
            _not_overlapping(where, name, t)
        outs.append(t)
        packed.append(_pack_heads(*_heads_tensor(where, name, t)))
    p = _problem(where, q, k, v, o, lse, causal, window, scale, q_len, kv_len, do=do, dq=outs[0], dk=outs[1],
                 dv=outs[2], workspace=workspace)
    _check_workspace(where, workspace)
    lib, index = _lib(), q.get_device()
    ws, nbytes = _ws(lib.pamm_attention_backward_workspace_size(p), q.device, workspace, where)
    _launch("pamm_attention_backward", index, lib.pamm_attention_backward, p, *packed, ws, nbytes,
            _stream_of(index))
    return tuple(outs)


# ------------------------------------------------------------------------ norm

def _row_major(where, name, t, n, d, dtype):
    """The leading dimension of an [n x d] tensor."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{where}: {name} must be a 2-D tensor with contiguous rows")
    if t.shape != (n, d):
        raise ValueError(f"{where}: {name} must have shape {(n, d)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    # a single row has no distance to the next
    return t.stride(0) if n > 1 else (d + 15) // 16 * 16


def _written_rows(where, name, t, n, d, dtype):
    ld = _row_major(where, name, t, n, d, dtype)
    if n > 1 and ld < d:
        raise ValueError(f"{where}: {name} is written and must not overlap itself, got strides {t.stride()}")
    return ld


def _rows_like(t):
    """Uninitialised rows of t's shape and dtype, a multiple of 16 bytes apart."""
    if t.is_contiguous() and t.shape[1] * t.element_size() % 16 == 0:
        return torch.empty_like(t)
    return _empty_rows(t.shape[0], t.shape[1], t.dtype, t.device)


def _vector(where, name, t, d, dtype):
    if t.dim() != 1 or t.shape[0] != d or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous {dtype} of shape {(d,)}, got {tuple(t.shape)} {t.dtype}")


def _norm_forward(where, x, weight, residual, eps, h, y, q, qscale, want_q, stream):
    if stream is not None:
        return _under(stream, where, x, _norm_forward, where, x, weight, residual, eps, h, y, q, qscale, want_q, None)
    if x.dim() != 2:
        raise ValueError(f"{where}: x must be a 2-D tensor with contiguous rows")
    n, d = x.shape
    dtype, device = x.dtype, x.device
    dt = _code(where, x)
    ldx = _row_major(where, "x", x, n, d, dtype)
    _vector(where, "weight", weight, d, dtype)
    _on_gpu(where, x=x, weight=weight, residual=residual, h=h, y=y, q=q, qscale=qscale)
    if residual is None:
        if h is not None:
            raise ValueError(f"{where}: h is x itself without a residual")
        h_out, ldh, ldr, rp, hp = x, 0, 0, None, None
    else:
        ldr = _row_major(where, "residual", residual, n, d, dtype)
        h_out = h if h is not None else _rows_like(x)
        ldh = _written_rows(where, "h", h_out, n, d, dtype)
        rp, hp = residual.data_ptr(), h_out.data_ptr()
    ldy = ldq = 0
    yp = qp = sp = None
    if want_q:
        if q is None:
            wide = (d + 7) // 8 * 8
            q = torch.empty((n, wide), dtype=torch.float8_e4m3fn, device=device)
            if wide != d:
                q = q[:, :d]
        ldq = _written_rows(where, "q", q, n, d, torch.float8_e4m3fn)
        if qscale is None:
            qscale = torch.empty(n, dtype=torch.float32, device=device)
        else:
            _vector(where, "qscale", qscale, n, torch.float32)
        qp, sp = q.data_ptr(), qscale.data_ptr()
    else:
        y = y if y is not None else _rows_like(x)
        ldy = _written_rows(where, "y", y, n, d, dtype)
        yp = y.data_ptr()
    rstd = torch.empty(n, dtype=torch.float32, device=device)
    index = x.get_device()
    _launch("pamm_add_rms_norm", index, _lib().pamm_add_rms_norm, x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), n, d,
            dt, eps, hp, ldh, yp, ldy, qp, ldq, sp, rstd.data_ptr(), _stream_of(index))
    return (q, qscale, h_out, rstd) if want_q else (y, h_out, rstd)


def add_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, h=None, y=None, stream=None):
    """h = x + residual (rounded to the dtype; x itself without a residual) and
    y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps) of each row.

    x, residual [n x d], weight [d], bf16 or fp32, rows a multiple of 16 bytes
    apart.  Returns (y, h, rstd [n] fp32); h may be written over x or
    residual (pass it as ``h``)."""
    return _norm_forward("add_rms_norm", x, weight, residual, eps, h, y, None, None, False, stream)


def add_rms_norm_fp8(x, weight, residual=None, *, eps: float = 1e-6, h=None, q=None, qscale=None, stream=None):
    """add_rms_norm with y in 8 bits: returns (q [n x d] float8_e4m3fn,
    qscale [n] fp32, h, rstd) with y ~ q * qscale[:, None].

    qscale is each row's largest |y| / 448 (at least 2^-126), the row-wise
    form an 8-bit matrix product takes; y / qscale is rounded once, to nearest
    even, for bf16 exactly as in the definition."""
    return _norm_forward("add_rms_norm_fp8", x, weight, residual, eps, h, None, q, qscale, True, stream)


def add_rms_norm_backward(dy, h, weight, rstd, *, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of add_rms_norm from dy, the gradient of y, its outputs h and
    rstd, and dh, the gradient that reaches h by the residual path.

    Returns (dx [n x d], the gradient of x and of residual alike,
    dweight [d] fp32).  dx may be dy or dh itself.  Bitwise deterministic."""
    where = "add_rms_norm_backward"
    if stream is not None:
        return _under(stream, where, h, add_rms_norm_backward, dy, h, weight, rstd, dh=dh, dx=dx, dweight=dweight,
                      workspace=workspace)
    if h.dim() != 2:
        raise ValueError(f"{where}: h must be a 2-D tensor with contiguous rows")
    n, d = h.shape
    dtype = h.dtype
    dt = _code(where, h)
    ldh = _row_major(where, "h", h, n, d, dtype)
    lddy = _row_major(where, "dy", dy, n, d, dtype)
    lddh = _row_major(where, "dh", dh, n, d, dtype) if dh is not None else 0
    _vector(where, "weight", weight, d, dtype)
    _vector(where, "rstd", rstd, n, torch.float32)
    _on_gpu(where, h=h, dy=dy, dh=dh, weight=weight, rstd=rstd, dx=dx, dweight=dweight, workspace=workspace)
    _check_workspace(where, workspace)
    dx = dx if dx is not None else _rows_like(h)
    lddx = _written_rows(where, "dx", dx, n, d, dtype)
    if dweight is None:
        dweight = torch.empty(d, dtype=torch.float32, device=h.device)
    else:
        _vector(where, "dweight", dweight, d, torch.float32)
    lib, index = _lib(), h.get_device()
    ws, nbytes = _ws(lib.pamm_add_rms_norm_backward_workspace_size(n, d, dt), h.device, workspace, where)
    _launch("pamm_add_rms_norm_backward", index, lib.pamm_add_rms_norm_backward, dy.data_ptr(), lddy, h.data_ptr(),
            ldh, weight.data_ptr(), rstd.data_ptr(), dh.data_ptr() if dh is not None else None, lddh, n, d, dt,
            dx.data_ptr(), lddx, dweight.data_ptr(), ws, nbytes, _stream_of(index))
    return dx, dweight


# -------------------------------------------------------------------- clipping

def _grad_layout(where, name, t):
    """(rows, cols, ld): one row for any dense layout (element order does not
    matter to a sum of squares or a scaling), else 2-D rows ld apart."""
    n = t.numel()
    if t.is_contiguous() or n <= 1:
        return 1, n, n
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t.shape[0], t.shape[1], t.stride(0)
    need = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride != need:
            raise ValueError(f"{where}: {name} must be dense or 2-D with contiguous rows, got strides {t.stride()} "
                             f"for shape {tuple(t.shape)}")
        need *= size
    return 1, n, n


def clip_grad_norm(grads, max_norm=None, *, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """The 2-norm of all gradients together (a 0-D fp32 tensor on the GPU), and
    their scaling by min(1, max_norm / (norm + eps)), in place or into ``out``.

    grads: a list of bf16 and fp32 tensors on one GPU, dense or 2-D with
    contiguous rows (such as the padded rows of a weight gradient); None
    entries are skipped.  out: as many tensors of the same shapes, bf16 or
    fp32 (for instance fp32 copies for an optimizer).  max_norm None, or
    infinity without out: the norm alone; out is always written whole.  Squares
    are summed in 64 bits; a norm under the limit leaves gradients in place
    untouched.  Nothing waits for the GPU."""
    where = "clip_grad_norm"
    if isinstance(grads, torch.Tensor):
        grads = [grads]
        out = [out] if isinstance(out, torch.Tensor) else out
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{where}: {len(grads)} gradients and {len(outs)} outputs")
    if out is not None and max_norm is None:
        raise ValueError(f"{where}: out needs a max_norm")
    first = next((g for g in grads if g is not None), None)
    if first is None:
        raise ValueError(f"{where}: no gradient given")
    if stream is not None:
        return _under(stream, where, first, clip_grad_norm, grads, max_norm, eps=eps, out=out, workspace=workspace)
    index, device, codes, packed = first.get_device(), first.device, _CODES, []
    for i, (g, o) in enumerate(zip(grads, outs)):
        if g is None:
            continue
        if index < 0 or g.get_device() != index:
            raise ValueError(f"{where}: gradient {i} must be on one GPU with the others, got device {g.device}")
        code = codes.get(g.dtype)
        if code is None:
            _code(where, g)
        if o is g:
            if g.is_contiguous():
                n, p = g.numel(), g.data_ptr()
                packed.append(_pack_grad(p, p, 1, n, n, n, code, code))
            else:
                rows, cols, ld = _grad_layout(where, f"gradient {i}", g)
                packed.append(_pack_grad(g.data_ptr(), g.data_ptr(), rows, cols, ld, ld, code, code))
            continue
        if o is None or o.shape != g.shape or o.get_device() != index:
            raise ValueError(f"{where}: output {i} must have shape {tuple(g.shape)} on {device}")
        code_o = codes.get(o.dtype)
        if code_o is None:
            _code(where, o)
        if g.is_contiguous() and o.is_contiguous():
            n = g.numel()
            packed.append(_pack_grad(g.data_ptr(), o.data_ptr(), 1, n, n, n, code, code_o))
            continue
        lay, lay_o = _grad_layout(where, f"gradient {i}", g), _grad_layout(where, f"output {i}", o)
        if (lay[0] == 1) != (lay_o[0] == 1) and g.dim() == 2 and (g.is_contiguous() or o.is_contiguous()):
            # one dense, one with padded rows: both as rows
            lay, lay_o = ((t.shape[0], t.shape[1], t.stride(0)) for t in (g, o))
        elif lay[:2] != lay_o[:2] or (lay[0] == 1 and g.stride() != o.stride()):
            raise ValueError(f"{where}: output {i} must be laid out as its gradient")
        packed.append(_pack_grad(g.data_ptr(), o.data_ptr(), lay[0], lay[1], lay[2], lay_o[2], code, code_o))
    # the library takes infinity as the norm alone, and as fp32 any number past its range is that
    limit = math.inf if max_norm is None else float(max_norm)
    if max_norm is not None and (out is not None or limit != math.inf):
        limit = min(limit, _FLT_MAX)
    count, arr = len(packed), b"".join(packed)
    if workspace is not None:
        _check_workspace(where, workspace)
        _on_gpu(where, gradients=first, workspace=workspace)
    norm = torch.empty((), dtype=torch.float32, device=device)
    lib = _lib()
    ws, nbytes = _ws(lib.pamm_clip_grad_norm_workspace_size(arr, count), device, workspace, where)
    try:
        _launch("pamm_clip_grad_norm", index, lib.pamm_clip_grad_norm, arr, count,
                limit, float(eps), norm.data_ptr(), ws, nbytes, _stream_of(index))
    except PammError as e:
        if e.status == 10:  # PAMM_ERR_OVERLAP
            raise ValueError(f"{where}: two gradients share memory that is written") from e
        raise
    return norm
