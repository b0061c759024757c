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
All calls are asynchronous on the current stream (or ``stream``).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (BF16, F32, _check, _dtype_code, _empty_rows, _on_gpu, _ptr, _rows, _stream_ptr, _check_workspace,
               load_library)

__all__ = ["attention", "attention_backward", "attention_workspace_size", "attention_backward_workspace_size",
           "add_rms_norm", "add_rms_norm_fp8", "add_rms_norm_backward", "clip_grad_norm", "MAX_HEAD_DIM"]

MAX_HEAD_DIM = 128

_i32, _i64, _f32, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_b", _i64), ("stride_s", _i64), ("stride_h", _i64)]


class _Attention(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("causal", _i32), ("batch", _i64), ("seq_q", _i64), ("seq_k", _i64),
                ("heads", _i64), ("heads_kv", _i64), ("head_dim", _i64), ("window", _i64), ("scale", _f32),
                ("q_len", _vp), ("kv_len", _vp), ("q", _Heads), ("k", _Heads), ("v", _Heads), ("o", _Heads),
                ("lse", _vp)]


class _Grad(ctypes.Structure):
    _fields_ = [("data", _vp), ("out", _vp), ("rows", _i64), ("cols", _i64), ("ld", _i64), ("ld_out", _i64),
                ("dtype", _i32), ("out_dtype", _i32)]


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


def _ws(nbytes, device, workspace, where):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"{where}: workspace needs {nbytes} bytes")
    return workspace, workspace.numel() * workspace.element_size()


class _on_device:
    """The tensors' GPU as the current one (nothing to do where it already is):
    kernels are launched on the device their memory and stream belong to."""

    def __init__(self, device):
        self.device, self.before = device.index, None

    def __enter__(self):
        now = torch.cuda.current_device()
        if self.device is not None and self.device != now:
            self.before = now
            torch.cuda.set_device(self.device)

    def __exit__(self, *exc):
        if self.before is not None:
            torch.cuda.set_device(self.before)


def _stream_of(stream, device):
    return _stream_ptr(stream if stream is not None else torch.cuda.current_stream(device))


# ------------------------------------------------------------------- attention

def _heads_tensor(where, name, t):
    if t.dim() != 4:
        raise ValueError(f"{where}: {name} must be 4-D [batch x sequence x heads x head_dim], "
                         f"got shape {tuple(t.shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{where}: {name} must have contiguous head rows (stride 1 in the last dimension)")


def _heads(t):
    return _Heads(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _lengths(where, name, t, batch, like):
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != batch:
        raise ValueError(f"{where}: {name} must have shape {(batch,)}, got {tuple(t.shape)}")
    if t.dtype != torch.int32:
        raise TypeError(f"{where}: {name} must be int32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    return t


def _problem(where, q, k, v, o, lse, causal, window, scale, q_len, kv_len):
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        if t is not None:
            _heads_tensor(where, name, t)
            if t.dtype != q.dtype:
                raise TypeError(f"{where}: q, k, v and o must share a dtype, got {q.dtype} and {t.dtype}")
    B, Sq, H, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"{where}: k and v must be [{B} x sequence x heads x {D}], got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{where}: {H} query heads do not share {Hkv} key/value heads evenly")
    _on_gpu(where, q=q, k=k, v=v, o=o, lse=lse, q_len=q_len, kv_len=kv_len)
    q_len = _lengths(where, "q_len", q_len, B, q)
    kv_len = _lengths(where, "kv_len", kv_len, B, q)
    if o is not None and tuple(o.shape) != (B, Sq, H, D):
        raise ValueError(f"{where}: o must have shape {(B, Sq, H, D)}, got {tuple(o.shape)}")
    if lse is not None:
        if tuple(lse.shape) != (B, H, Sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError(f"{where}: lse must be contiguous float32 of shape {(B, H, Sq)}")
    return _Attention(dtype=_dtype_code(q), causal=1 if causal else 0, batch=B, seq_q=Sq, seq_k=Sk, heads=H,
                      heads_kv=Hkv, head_dim=D, window=int(window or 0),
                      scale=float(1.0 / math.sqrt(max(D, 1)) if scale is None else scale),
                      q_len=q_len.data_ptr() if q_len is not None else None,
                      kv_len=kv_len.data_ptr() if kv_len is not None else None,
                      q=_heads(q), k=_heads(k), v=_heads(v))


def attention_workspace_size(q, k, *, causal=False) -> int:
    """Bytes of workspace ``attention`` needs for tensors of these shapes."""
    p = _problem("attention_workspace_size", q, k, k, None, None, causal, 0, None, None, None)
    return int(_lib().pamm_attention_workspace_size(ctypes.byref(p)))


def attention_backward_workspace_size(q, k, *, causal=False) -> int:
    """Bytes of workspace ``attention_backward`` needs for tensors of these shapes."""
    p = _problem("attention_backward_workspace_size", q, k, k, None, None, causal, 0, None, None, None)
    return int(_lib().pamm_attention_backward_workspace_size(ctypes.byref(p)))


def _not_overlapping(where, name, t):
    """A written tensor must give every element an address of its own."""
    need = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < need:
            raise ValueError(f"{where}: {name} is written and must not overlap itself, got strides {t.stride()} "
                             f"for shape {tuple(t.shape)}")
        need = stride * (size - 1) + need
    return t


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
    key has o = 0 and lse = -inf.  attention_backward takes both."""
    p = _problem("attention", q, k, v, o, lse, causal, window, scale, q_len, kv_len)
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _not_overlapping("attention", "o", o)
    if lse is None:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
    p.o, p.lse = _heads(o), lse.data_ptr()
    _check_workspace("attention", workspace)
    _on_gpu("attention", q=q, workspace=workspace)
    lib = _lib()
    with _on_device(q.device):
        ws, nbytes = _ws(lib.pamm_attention_workspace_size(ctypes.byref(p)), q.device, workspace, "attention")
        _check(lib.pamm_attention(ctypes.byref(p), _ptr(ws), nbytes, _stream_of(stream, q.device)), "pamm_attention")
    return o, lse


def attention_backward(do, q, k, v, o, lse, *, causal: bool = False, window: int = 0, scale=None, q_len=None,
                       kv_len=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of ``attention`` from do, the gradient of its o,
    and its outputs; the other arguments as they were given to it.

    The probabilities are recomputed from q, k and lse, so nothing of size
    Sq x Sk exists.  dk and dv are summed over the query heads that share
    them.  dq, dk and dv may be given (strided views, for instance of one
    packed gradient); they are written whole, with zeros past the lengths.
    Bitwise deterministic."""
    where = "attention_backward"
    p = _problem(where, q, k, v, o, lse, causal, window, scale, q_len, kv_len)
    _heads_tensor(where, "do", do)
    if tuple(do.shape) != tuple(q.shape) or do.dtype != q.dtype:
        raise ValueError(f"{where}: do must be {q.dtype} of shape {tuple(q.shape)}, got {tuple(do.shape)} {do.dtype}")
    outs = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            t = torch.empty(like.shape, dtype=like.dtype, device=like.device)
        else:
            _heads_tensor(where, name, t)
            if tuple(t.shape) != tuple(like.shape) or t.dtype != like.dtype:
                raise ValueError(f"{where}: {name} must be {like.dtype} of shape {tuple(like.shape)}, "
                                 f"got {tuple(t.shape)} {t.dtype}")
            _not_overlapping(where, name, t)
        outs.append(t)
    p.o, p.lse = _heads(o), lse.data_ptr()
    _check_workspace(where, workspace)
    _on_gpu(where, q=q, do=do, dq=outs[0], dk=outs[1], dv=outs[2], workspace=workspace)
    lib = _lib()
    h = [_heads(t) for t in (do, *outs)]
    with _on_device(q.device):
        ws, nbytes = _ws(lib.pamm_attention_backward_workspace_size(ctypes.byref(p)), q.device, workspace, where)
        _check(lib.pamm_attention_backward(ctypes.byref(p), ctypes.byref(h[0]), ctypes.byref(h[1]), ctypes.byref(h[2]),
                                           ctypes.byref(h[3]), _ptr(ws), nbytes, _stream_of(stream, q.device)),
               "pamm_attention_backward")
    return tuple(outs)


# ------------------------------------------------------------------------ norm

def _row_major(where, name, t, n, d, dtype):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{where}: {name} must be a 2-D tensor with contiguous rows")
    if tuple(t.shape) != (n, d):
        raise ValueError(f"{where}: {name} must have shape {(n, d)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    # a single row has no distance to the next
    return t.stride(0) if n > 1 else _padded(d, t.element_size())


def _padded(d, size):
    per = max(1, (8 if size == 1 else 16) // size)
    return (d + per - 1) // per * per


def _vector(where, name, t, d, dtype):
    if t.dim() != 1 or t.shape[0] != d or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous {dtype} of shape {(d,)}, got {tuple(t.shape)} {t.dtype}")


def _norm_forward(where, x, weight, residual, eps, h, y, q, qscale, want_q, stream):
    n, d, _ = _rows(x, "x")
    dt = _dtype_code(x)
    ldx = _row_major(where, "x", x, n, d, x.dtype)
    _vector(where, "weight", weight, d, x.dtype)
    _on_gpu(where, x=x, weight=weight, residual=residual, h=h, y=y, q=q, qscale=qscale)
    ldr = _row_major(where, "residual", residual, n, d, x.dtype) if residual is not None else 0
    if h is not None and residual is None:
        raise ValueError(f"{where}: h is x itself without a residual")
    if residual is None:
        h_out, ldh = x, 0
    else:
        h_out = h if h is not None else _empty_rows(n, d, x.dtype, x.device)
        ldh = _row_major(where, "h", h_out, n, d, x.dtype)
        _not_overlapping(where, "h", h_out)
    ldy = ldq = 0
    if want_q:
        if q is None:
            q = torch.empty((n, _padded(d, 1)), dtype=torch.float8_e4m3fn, device=x.device)[:, :d]
        ldq = _row_major(where, "q", q, n, d, torch.float8_e4m3fn)
        _not_overlapping(where, "q", q)
        if qscale is None:
            qscale = torch.empty(n, dtype=torch.float32, device=x.device)
        _vector(where, "qscale", qscale, n, torch.float32)
    else:
        y = y if y is not None else _empty_rows(n, d, x.dtype, x.device)
        ldy = _row_major(where, "y", y, n, d, x.dtype)
        _not_overlapping(where, "y", y)
    rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    with _on_device(x.device):
        st = _lib().pamm_add_rms_norm(
            _ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), n, d, dt, float(eps),
            _ptr(h_out) if residual is not None else None, ldh, None if want_q else _ptr(y), ldy,
            _ptr(q) if want_q else None, ldq, _ptr(qscale) if want_q else None, _ptr(rstd),
            _stream_of(stream, x.device))
        _check(st, "pamm_add_rms_norm")
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
    form an 8-bit matrix product takes; y is rounded once, from fp32."""
    return _norm_forward("add_rms_norm_fp8", x, weight, residual, eps, h, None, q, qscale, True, stream)


def add_rms_norm_backward(dy, h, weight, rstd, *, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of add_rms_norm from dy, the gradient of y, its outputs h and
    rstd, and dh, the gradient that reaches h by the residual path.

    Returns (dx [n x d], the gradient of x and of residual alike,
    dweight [d] fp32).  dx may be dy or dh itself.  Bitwise deterministic."""
    where = "add_rms_norm_backward"
    n, d, _ = _rows(h, "h")
    dt = _dtype_code(h)
    ldh = _row_major(where, "h", h, n, d, h.dtype)
    lddy = _row_major(where, "dy", dy, n, d, h.dtype)
    lddh = _row_major(where, "dh", dh, n, d, h.dtype) if dh is not None else 0
    _vector(where, "weight", weight, d, h.dtype)
    _vector(where, "rstd", rstd, n, torch.float32)
    _on_gpu(where, h=h, dy=dy, dh=dh, weight=weight, rstd=rstd, dx=dx, dweight=dweight, workspace=workspace)
    _check_workspace(where, workspace)
    dx = dx if dx is not None else _empty_rows(n, d, h.dtype, h.device)
    lddx = _row_major(where, "dx", dx, n, d, h.dtype)
    _not_overlapping(where, "dx", dx)
    if dweight is None:
        dweight = torch.empty(d, dtype=torch.float32, device=h.device)
    _vector(where, "dweight", dweight, d, torch.float32)
    lib = _lib()
    with _on_device(h.device):
        ws, nbytes = _ws(lib.pamm_add_rms_norm_backward_workspace_size(n, d, dt), h.device, workspace, where)
        _check(lib.pamm_add_rms_norm_backward(_ptr(dy), lddy, _ptr(h), ldh, _ptr(weight), _ptr(rstd), _ptr(dh), lddh,
                                              n, d, dt, _ptr(dx), lddx, _ptr(dweight), _ptr(ws), nbytes,
                                              _stream_of(stream, h.device)), "pamm_add_rms_norm_backward")
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


def _written_apart(where, grads, outs, layouts, out_layouts):
    """No written range may meet another tensor's: each element is scaled once."""
    spans = []
    for i, (g, o) in enumerate(zip(grads, outs)):
        rows, cols, ld = out_layouts[i]
        if rows * cols:
            spans.append((o.data_ptr(), o.data_ptr() + ((rows - 1) * ld + cols) * o.element_size(), i, True))
        if o is not g and layouts[i][0] * layouts[i][1]:
            rows, cols, ld = layouts[i]
            spans.append((g.data_ptr(), g.data_ptr() + ((rows - 1) * ld + cols) * g.element_size(), i, False))
    spans.sort()
    active = []  # earlier spans that reach past the current one's start
    for span in spans:
        b1, _, j, w1 = span
        active = [s for s in active if s[1] > b1]
        for b0, _, i, w0 in active:
            if not (w0 or w1):
                continue
            # columns of one wider matrix interleave without meeting
            a, b = (outs if w0 else grads)[i], (outs if w1 else grads)[j]
            la, lb = (out_layouts if w0 else layouts)[i], (out_layouts if w1 else layouts)[j]
            size = a.element_size()
            if la[0] > 1 and lb[0] > 1 and la[2] == lb[2] and size == b.element_size() and (b1 - b0) % size == 0:
                shift = (b1 - b0) // size % la[2]
                if shift >= la[1] and shift + lb[1] <= la[2]:
                    continue
            raise ValueError(f"{where}: gradients {i} and {j} share memory that is written")
        active.append(span)


def clip_grad_norm(grads, max_norm=None, *, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """The 2-norm of all gradients together (a 0-D fp32 tensor on the GPU), and
    their scaling by min(1, max_norm / (norm + eps)), in place or into ``out``.

    grads: a list of bf16 and fp32 tensors on one GPU, dense or 2-D with
    contiguous rows (such as the padded rows of a weight gradient); None
    entries are skipped.  out: as many tensors of the same shapes, bf16 or
    fp32 (for instance fp32 copies for an optimizer).  max_norm None: the norm
    alone.  Squares are summed in 64 bits; a norm under the limit leaves
    gradients in place untouched.  Nothing waits for the GPU."""
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
    pairs = [(g, o) for g, o in zip(grads, outs) if g is not None]
    if not pairs:
        raise ValueError(f"{where}: no gradient given")
    grads, outs = [g for g, _ in pairs], [o for _, o in pairs]
    device = grads[0].device
    flat, layouts, out_layouts = [], [], []
    for i, (g, o) in enumerate(pairs):
        if not g.is_cuda or g.device != device:
            raise ValueError(f"{where}: gradient {i} must be on one GPU with the others, got device {g.device}")
        lay = _grad_layout(where, f"gradient {i}", g)
        layouts.append(lay)
        code = _dtype_code(g)
        if o is g:
            lay_o, code_o = lay, code
        else:
            if o is None or o.shape != g.shape or o.device != device:
                raise ValueError(f"{where}: output {i} must have shape {tuple(g.shape)} on {device}")
            lay_o, code_o = _grad_layout(where, f"output {i}", o), _dtype_code(o)
            if g.stride() != o.stride() and (lay[0] == 1) != (lay_o[0] == 1):
                # one dense, one with padded rows: describe both as rows
                if g.dim() == 2 and g.is_contiguous():
                    lay = layouts[-1] = (g.shape[0], g.shape[1], g.shape[1])
                elif o.dim() == 2 and o.is_contiguous():
                    lay_o = (o.shape[0], o.shape[1], o.shape[1])
                else:
                    raise ValueError(f"{where}: output {i} must be laid out as its gradient")
            elif lay[0] == 1 and g.stride() != o.stride() and not (g.is_contiguous() and o.is_contiguous()):
                raise ValueError(f"{where}: output {i} must be laid out as its gradient")
        out_layouts.append(lay_o)
        flat.append((g.data_ptr(), o.data_ptr(), lay[0], lay[1], lay[2], lay_o[2], code, code_o))
    if max_norm is not None:
        _written_apart(where, grads, outs, layouts, out_layouts)
    arr = (_Grad * len(flat))(*flat)
    _check_workspace(where, workspace)
    _on_gpu(where, grads=grads[0], workspace=workspace)
    norm = torch.empty((), dtype=torch.float32, device=device)
    lib = _lib()
    with _on_device(device):
        ws, nbytes = _ws(lib.pamm_clip_grad_norm_workspace_size(arr, len(flat)), device, workspace, where)
        _check(lib.pamm_clip_grad_norm(arr, len(flat), math.inf if max_norm is None else float(max_norm), float(eps),
                                       _ptr(norm), _ptr(ws), nbytes, _stream_of(stream, device)),
               "pamm_clip_grad_norm")
    return norm
