"""A cache of keys and values in 8 bits, with a scale for each block of tokens
and head, and attention over it.

Thin binding over the C ABI of ``include/pamm_cache.h`` (the same
``libpamm.so``), in the manner of block_ops: PyTorch supplies device memory and
the stream, every step runs in the library's HIP kernels, there is no CPU
fallback, and all calls are asynchronous on the current stream or ``stream``.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _check_workspace, _on_gpu, load_library
from .block_ops import (MAX_HEAD_DIM, _HEADS, _apart, _code, _heads_tensor, _launch, _lengths, _not_overlapping, _pack_attention,
                        _pack_heads, _stream_of, _under, _ws)

__all__ = ["CacheFP8", "cache_append_fp8", "attention_fp8", "attention_fp8_workspace_size"]

_sz, _vp, _i64, _i32 = ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

# pamm_cache8_t
_pack_cache = struct.Struct("@i4x5q" + 6 * _HEADS).pack

_CACHE_EXPORTS = {
    "pamm_cache8_append": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, _i32, _vp]),
    "pamm_cache8_attention_workspace_size": (_sz, [_vp, _vp]),
    "pamm_cache8_attention": (ctypes.c_int, [_vp, _vp, _vp, _sz, _vp]),
}
_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = load_library()
        for name, (res, args) in _CACHE_EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _bound = lib
    return _bound


class CacheFP8(NamedTuple):
    """Keys and values [B x room x Hkv x D] in 8 bits (float8_e4m3fn), their
    scales [B x room // block x Hkv] in fp32, and the tails [B x block x Hkv x D]
    in the type of the queries, where the tokens of each sequence's last,
    partial block wait; block (32, 64 or 128) is the tails' length.  Token j
    stands for k[b, j, h] * k_scale[b, j // block, h]; k is the nearest to
    448 x / max|x|, k_scale is max|x| / 448, over a block of one head."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_tail: torch.Tensor
    v_tail: torch.Tensor

    @classmethod
    def empty(cls, batch: int, room: int, heads_kv: int, head_dim: int, *, block: int = 64, device="cuda",
              dtype=torch.bfloat16):
        """A cache for ``room`` tokens a sequence, nothing written: one head's
        tokens lie side by side, so that single queries read long runs."""
        if block not in (32, 64, 128):
            raise ValueError(f"CacheFP8: block must be 32, 64 or 128, got {block}")
        if head_dim % 16 or not 0 < head_dim <= MAX_HEAD_DIM:
            raise ValueError(f"CacheFP8: head_dim must be a multiple of 16 up to {MAX_HEAD_DIM}, got {head_dim}")

        def heads(rows, dt):
            return torch.empty(batch, heads_kv, rows, head_dim, dtype=dt, device=device).transpose(1, 2)

        def scales():
            return torch.empty(batch, heads_kv, room // block, dtype=torch.float32, device=device).transpose(1, 2)

        return cls(heads(room, torch.float8_e4m3fn), heads(room, torch.float8_e4m3fn), scales(), scales(),
                   heads(block, dtype), heads(block, dtype))


_F8, _F32 = torch.float8_e4m3fn, torch.float32


def _cache(where, c, written):
    """The checked cache as a packed pamm_cache8_t."""
    k, v, ks, vs, kt, vt = c
    shape, tail, dtype = k.shape, kt.shape, kt.dtype
    kst, vst, kts, vts = k.stride(), v.stride(), kt.stride(), vt.stride()
    if len(shape) != 4 or len(tail) != 4 or len(vst) != 4 or len(vts) != 4 or not kst[3] == vst[3] == kts[3] == vts[3] == 1:
        for name, t in (("k", k), ("v", v), ("k_tail", kt), ("v_tail", vt)):
            _heads_tensor(where, f"cache.{name}", t)
    B, room, H, D = shape
    block = tail[1]
    if k.dtype != _F8 or v.dtype != _F8:
        raise TypeError(f"{where}: the cache's k and v must be float8_e4m3fn, got {k.dtype} and {v.dtype}")
    if v.shape != shape:
        raise ValueError(f"{where}: the cache's k and v must share a shape, got {tuple(k.shape)} and {tuple(v.shape)}")
    if block not in (32, 64, 128):
        raise ValueError(f"{where}: the cache's tails must hold a block of 32, 64 or 128 tokens, got {block}")
    if tail != (B, block, H, D) or vt.shape != tail:
        raise ValueError(f"{where}: the cache's tails must have shape {(B, block, H, D)}, got {tuple(kt.shape)} and "
                         f"{tuple(vt.shape)}")
    if vt.dtype != dtype:
        raise TypeError(f"{where}: the cache's tails must share a dtype, got {kt.dtype} and {vt.dtype}")
    if ks.dtype != _F32 or vs.dtype != _F32:
        raise TypeError(f"{where}: the cache's k_scale and v_scale must be float32, got {ks.dtype} and {vs.dtype}")
    blocks, kss, vss = room // block, ks.shape, vs.shape
    # more blocks than the rows in view: of a cache whose k and v are sliced
    for name, n in (("k_scale", kss), ("v_scale", vss)):
        if len(n) != 3 or n[0] != B or n[2] != H or n[1] < blocks:
            raise ValueError(f"{where}: the cache's {name} must have shape {(B, blocks, H)}, got {tuple(n)}")
    kst3, vst3 = ks.stride(), vs.stride()
    if written and not (_apart(kst, (room, H), D) and _apart(vst, (room, H), D) and _apart(kts, (block, H), D)
                        and _apart(vts, (block, H), D) and _apart(kst3, (kss[1], H), 1) and _apart(vst3, (vss[1], H), 1)):
        for name, t in zip(c._fields, c):
            _not_overlapping(where, f"cache.{name}", t)
    return _pack_cache(_code(where, kt), B, room, H, D, block, k.data_ptr(), *kst[:3], v.data_ptr(), *vst[:3],
                       ks.data_ptr(), *kst3, vs.data_ptr(), *vst3, kt.data_ptr(), *kts[:3], vt.data_ptr(), *vts[:3])


def _one_gpu(where, cache, **tensors):
    """The GPU that all tensors are on."""
    index = cache[0].get_device()
    if index >= 0:
        for t in cache:
            if t.get_device() != index:
                break
        else:
            for t in tensors.values():
                if t is not None and t.get_device() != index:
                    break
            else:
                return index
    _on_gpu(where, **tensors, **{f"cache_{n}": t for n, t in zip(cache._fields, cache)})  # says which


def cache_append_fp8(cache: CacheFP8, k, v, lengths, *, new_len=None, advance: bool = True, stream=None):
    """Appends k and v [B x n x Hkv x D] (of the tails' dtype, any strides of the
    outer dimensions) behind the lengths[b] tokens of each sequence ([B] int32):
    all n of them, or the first new_len[b] ([B] int32).

    Blocks that become whole are put into 8 bits, 448 x / max|x| over the block,
    with a scale of max|x| / 448; the tokens behind them wait in the tail as they
    are.  What the cache holds is thus the same whatever chunks its tokens came in.
    What is not finite becomes NaN in 8 bits and does not count for the scale.
    lengths becomes the new lengths (with advance; else it is left).  Tokens
    that do not fit the cache's room are dropped, as the lengths are known on
    the GPU alone."""
    where = "cache_append_fp8"
    if stream is not None:
        return _under(stream, where, k, cache_append_fp8, cache, k, v, lengths, new_len=new_len, advance=advance)
    kh, vh = _heads_tensor(where, "k", k), _heads_tensor(where, "v", v)
    c = _cache(where, cache, True)
    B, _, H, D = cache.k.shape
    if k.shape != v.shape or (k.shape[0], k.shape[2], k.shape[3]) != (B, H, D):
        raise ValueError(f"{where}: k and v must be [{B} x tokens x {H} x {D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if k.dtype != cache.k_tail.dtype or v.dtype != k.dtype:
        raise TypeError(f"{where}: k and v must be {cache.k_tail.dtype}, got {k.dtype} and {v.dtype}")
    if lengths is None:
        raise ValueError(f"{where}: lengths are needed")
    at, new = _lengths(where, "lengths", lengths, B), _lengths(where, "new_len", new_len, B)
    index = _one_gpu(where, cache, k=k, v=v, lengths=lengths, new_len=new_len)
    _launch("pamm_cache8_append", index, _lib().pamm_cache8_append, c, _pack_heads(*kh), _pack_heads(*vh), k.shape[1],
            new, at, int(bool(advance)), _stream_of(index))


def _attention(where, q, cache, kv_len, causal, window, scale, q_len, o, lse, **others):
    """The GPU, and the checked arguments as a packed pamm_attention_t and pamm_cache8_t."""
    qh = _heads_tensor(where, "q", q)
    oh = _heads_tensor(where, "o", o) if o is not None else (0, 0, 0, 0)
    c = _cache(where, cache, False)
    B, Sq, H, D = q.shape
    Bk, room, Hkv, Dk = cache.k.shape
    if (Bk, Dk) != (B, D):
        raise ValueError(f"{where}: q {tuple(q.shape)} does not fit a cache of {tuple(cache.k.shape)}")
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{where}: {H} query heads do not share {Hkv} key/value heads evenly")
    if q.dtype != cache.k_tail.dtype or (o is not None and o.dtype != q.dtype):
        raise TypeError(f"{where}: q, o and the cache's tails must share a dtype, got {q.dtype}, "
                        f"{o.dtype if o is not None else None} and {cache.k_tail.dtype}")
    if o is not None and o.shape != q.shape:
        raise ValueError(f"{where}: o must have shape {(B, Sq, H, D)}, got {tuple(o.shape)}")
    if lse is not None and (lse.shape != (B, H, Sq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError(f"{where}: lse must be contiguous float32 of shape {(B, H, Sq)}")
    lengths = _lengths(where, "q_len", q_len, B), _lengths(where, "kv_len", kv_len, B)
    index = _one_gpu(where, cache, q=q, kv_len=kv_len, q_len=q_len, o=o, lse=lse, **others)
    none = (0, 0, 0, 0)
    return index, _pack_attention(_code(where, q), 1 if causal else 0, B, Sq, room, H, Hkv, D, int(window or 0),
                           1.0 / math.sqrt(max(D, 1)) if scale is None else float(scale), *lengths, *qh, *none, *none,
                           *oh, lse.data_ptr() if lse is not None else 0), c


def attention_fp8_workspace_size(q, cache: CacheFP8, kv_len=None) -> int:
    """Bytes of workspace ``attention_fp8`` needs for tensors of these shapes."""
    _, a, c = _attention("attention_fp8_workspace_size", q, cache, kv_len, False, 0, None, None, None, None)
    return int(_lib().pamm_cache8_attention_workspace_size(a, c))


def attention_fp8(q, cache: CacheFP8, kv_len, *, causal: bool = False, window: int = 0, scale=None, q_len=None, o=None,
                  lse=None, workspace=None, stream=None):
    """``attention`` of q [B x Sq x H x D] over a cache in 8 bits, with kv_len [B]
    int32 tokens in each sequence (None: the cache's rows are all valid; those
    of a last, partial block are the tail's).  These have to be the cache's own
    lengths: the tail holds the tokens behind its last whole block, so a length may
    be lowered (to take the last tokens back) as far as the end of that
    block, but a prefix that ends before it cannot be looked at.  Scales have to be
    positive, normal numbers, as cache_append_fp8 writes them.  Masks, heads, results (o, lse)
    and splitting over the device are those of ``attention``.

    Products of the 8-bit values are exact, their scales are applied in 32
    bits; in bf16 each probability times the values' scale is rounded once, to
    bf16, or to two bf16 parts where up to 32 query rows (Sq x H / Hkv) share a
    key/value head.
    cache.k and cache.v may be sliced to the rows in use.  For serving: there
    is no backward pass.  o and lse, where given, must not share memory with
    the inputs."""
    where = "attention_fp8"
    if stream is not None:
        return _under(stream, where, q, attention_fp8, q, cache, kv_len, causal=causal, window=window, scale=scale,
                      q_len=q_len, o=o, lse=lse, workspace=workspace)
    _heads_tensor(where, "q", q)
    if o is None:
        o = torch.empty_like(q)
    else:
        _heads_tensor(where, "o", o)
        _not_overlapping(where, "o", o)
    if lse is None:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
    index, a, c = _attention(where, q, cache, kv_len, causal, window, scale, q_len, o, lse, workspace=workspace)
    _check_workspace(where, workspace)
    lib = _lib()
    ws, nbytes = _ws(lib.pamm_cache8_attention_workspace_size(a, c), q.device, workspace, where)
    _launch("pamm_cache8_attention", index, lib.pamm_cache8_attention, a, c, ws, nbytes, _stream_of(index))
    return o, lse
