"""Host-side checks of include/pamm_cache.h and its binding (no GPU needed, no
kernel launched): exports, refusals, workspace sizes."""
import ctypes
import math
import os
import re

import pytest
import torch

import activation_compression_pamm_amd as pamm
from activation_compression_pamm_amd import cache_ops as ops
from activation_compression_pamm_amd.block_ops import _Attention, _Heads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EUNSUP, EHIP, EVALUE, ETOOLARGE = range(10)
FAKE = 0x10000  # an aligned, never-dereferenced address


class Cache8(ctypes.Structure):
    """pamm_cache8_t"""
    _l = ctypes.c_int64
    _fields_ = [("dtype", ctypes.c_int32), ("batch", _l), ("room", _l), ("heads_kv", _l), ("head_dim", _l), ("block", _l),
                ("k", _Heads), ("v", _Heads), ("k_scale", _Heads), ("v_scale", _Heads), ("k_tail", _Heads),
                ("v_tail", _Heads)]


def cache(**kw):
    d = dict(dtype=1, batch=2, room=640, heads_kv=2, head_dim=64, block=32)
    d.update(kw)
    c = Cache8(**d)
    for n, h in (("k", _Heads(FAKE, 640 * 128, 128, 64)), ("k_scale", _Heads(FAKE, 40, 2, 1)),
                 ("k_tail", _Heads(FAKE, 32 * 128, 128, 64))):
        for name in (n, "v" + n[1:]):
            if name not in kw:
                setattr(c, name, h)
    return c


def problem(**kw):
    d = dict(dtype=1, causal=1, batch=2, seq_q=3, seq_k=640, heads=4, heads_kv=2, head_dim=64, window=0, scale=0.125,
             lse=FAKE, kv_len=FAKE)
    d.update(kw)
    p = _Attention(**d)
    for n in ("q", "o"):
        if n not in kw:
            setattr(p, n, _Heads(FAKE, 3 * 256, 256, 64))
    return p


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pamm_cache.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(pamm_[a-z_0-9]+)\s*\(", text))) == sorted(ops._CACHE_EXPORTS)
    for name in ops._CACHE_EXPORTS:
        assert hasattr(lib, name)
    for name in ops.__all__:
        assert name in pamm.__all__ and callable(getattr(pamm, name))


def test_the_packed_struct_is_the_declared_one():
    raw = ops._pack_cache(*range(1, 31))
    assert len(raw) == ctypes.sizeof(Cache8)
    c = Cache8.from_buffer_copy(raw)
    assert (c.dtype, c.batch, c.block, c.k.data, c.v.stride_b, c.v_scale.stride_h, c.v_tail.stride_h) == (1, 2, 6, 7, 12, 22, 30)


BAD = [(dict(dtype=2), EDTYPE), (dict(batch=-1), ESHAPE), (dict(room=-1), ESHAPE), (dict(room=1 << 30), ESHAPE),
       (dict(heads_kv=0), ESHAPE), (dict(head_dim=0), ESHAPE), (dict(head_dim=144), ESHAPE), (dict(head_dim=56), EALIGN),
       (dict(block=0), EVALUE), (dict(block=48), EVALUE), (dict(block=256), EVALUE), (dict(block=-32), EVALUE),
       (dict(k=_Heads(None, 1 << 16, 128, 64)), ENULL), (dict(v=_Heads(FAKE + 8, 1 << 16, 128, 64)), EALIGN),
       (dict(k=_Heads(FAKE, 1 << 16, 128, 40)), EALIGN), (dict(v=_Heads(FAKE, -16, 128, 64)), ESHAPE),
       (dict(k=_Heads(FAKE, 1 << 42, 128, 64)), ESHAPE), (dict(k=_Heads(FAKE, 1 << 36, 1 << 25, 64)), EUNSUP),
       (dict(k_tail=_Heads(None, 4096, 128, 64)), ENULL), (dict(v_tail=_Heads(FAKE, 4096, 128, 60)), EALIGN),
       (dict(k_scale=_Heads(None, 40, 2, 1)), ENULL), (dict(v_scale=_Heads(FAKE + 2, 40, 2, 1)), EALIGN),
       (dict(k_scale=_Heads(FAKE, -1, 2, 1)), ESHAPE), (dict(k_scale=_Heads(FAKE, 1 << 50, 2, 1)), ESHAPE)]


@pytest.mark.parametrize("kw,status", BAD, ids=[str(i) for i in range(len(BAD))])
def test_refused_caches(lib, kw, status):
    c, h = cache(**kw), ctypes.byref(_Heads(FAKE, 384, 128, 64))
    assert lib.pamm_cache8_append(ctypes.byref(c), h, h, 3, None, FAKE, 1, None) == status
    same = {n: kw[n] for n in ("dtype", "batch", "heads_kv", "head_dim") if n in kw}
    got = lib.pamm_cache8_attention(ctypes.byref(problem(**same)), ctypes.byref(c), FAKE, 1 << 30, None)
    assert got == status or (status == ESHAPE and got in (ESHAPE, EALIGN))


def test_append_validation(lib):
    def call(c=None, k=_Heads(FAKE, 384, 128, 64), v=_Heads(FAKE, 384, 128, 64), n=3, new=None, lengths=FAKE, advance=1):
        ref = lambda x: ctypes.byref(x) if x is not None else None
        return lib.pamm_cache8_append(ctypes.byref(c or cache()), ref(k), ref(v), n, new, lengths, advance, None)

    assert lib.pamm_cache8_append(None, None, None, 3, None, FAKE, 1, None) == ENULL
    assert call(k=None) == ENULL and call(v=None) == ENULL and call(lengths=None) == ENULL
    assert call(n=-1) == ESHAPE and call(n=1 << 31) == ESHAPE and call(advance=2) == EVALUE
    assert call(new=FAKE + 2) == EALIGN and call(lengths=FAKE + 1) == EALIGN
    assert call(k=_Heads(FAKE + 4, 384, 128, 64)) == EALIGN and call(v=_Heads(FAKE, 384, -8, 64)) == ESHAPE
    # nothing to do is no error, and no launch
    assert call(n=0) == OK and call(c=cache(batch=0)) == OK


def test_attention_validation(lib):
    def call(p, c=None, ws=FAKE, n=1 << 30):
        return lib.pamm_cache8_attention(ctypes.byref(p), ctypes.byref(c or cache()), ws, n, None)

    size = lambda p, c=None: lib.pamm_cache8_attention_workspace_size(ctypes.byref(p), ctypes.byref(c or cache()))
    assert lib.pamm_cache8_attention(None, None, None, 0, None) == ENULL
    assert lib.pamm_cache8_attention_workspace_size(None, None) == 0
    assert call(problem(dtype=0)) == EDTYPE and call(problem(batch=3)) == ESHAPE and call(problem(heads_kv=4)) == ESHAPE
    assert call(problem(head_dim=32)) == ESHAPE and call(problem(seq_k=641)) == ESHAPE
    assert call(problem(heads=5)) == ESHAPE and call(problem(scale=math.nan)) == EVALUE
    assert call(problem(window=-1)) == EVALUE and call(problem(window=4, causal=0)) == EVALUE
    assert call(problem(q=_Heads(None, 768, 256, 64))) == ENULL and call(problem(o=_Heads(FAKE + 2, 768, 256, 64))) == EALIGN
    assert call(problem(lse=None)) == ENULL and call(problem(kv_len=FAKE + 2)) == EALIGN
    p, c = problem(seq_k=8192), cache(room=8192)  # long enough to be cut into parts
    need = size(p, c)
    assert need > 0 and need % 256 == 0 and size(problem(seq_k=32)) == 0
    assert call(p, c, ws=None) == EWS and call(p, c, n=need - 1) == EWS and call(p, c, ws=FAKE + 16) == EALIGN
    assert call(problem(batch=0), cache(batch=0)) == OK and call(problem(seq_q=0)) == OK


def tensors(B=2, room=128, H=2, D=32, **kw):
    return pamm.CacheFP8.empty(B, room, H, D, device="cpu", dtype=torch.float32, **kw)


def test_empty_cache():
    c = tensors(3, 130, 4, 48, block=64)
    assert c.k.shape == c.v.shape == (3, 130, 4, 48) and c.k.dtype == torch.float8_e4m3fn and c.k.stride(1) == 48
    assert c.k_scale.shape == (3, 2, 4) and c.k_tail.shape == (3, 64, 4, 48) and c.v_tail.dtype == torch.float32
    for kw in (dict(block=48), dict(D=24), dict(D=144), dict(D=0)):
        with pytest.raises(ValueError, match="CacheFP8"):
            tensors(**kw)


def test_arguments_are_checked_before_the_gpu_is_asked():
    c, n = tensors(), torch.zeros(2, dtype=torch.int32)
    x, q = torch.zeros(2, 3, 2, 32), torch.zeros(2, 3, 4, 32)
    half = c._replace(k_tail=c.k_tail.bfloat16(), v_tail=c.v_tail.bfloat16())
    cases = [
        (ValueError, "k and v must be", lambda: pamm.cache_append_fp8(c, x[:1], x[:1], n)),
        (ValueError, "k and v must be", lambda: pamm.cache_append_fp8(c, x, x[:, :2], n)),
        (TypeError, "k and v must be", lambda: pamm.cache_append_fp8(c, x.bfloat16(), x.bfloat16(), n)),
        (TypeError, "k and v must be", lambda: pamm.cache_append_fp8(half, x, x, n)),
        (ValueError, "lengths", lambda: pamm.cache_append_fp8(c, x, x, None)),
        (ValueError, "lengths", lambda: pamm.cache_append_fp8(c, x, x, n[:1])),
        (TypeError, "lengths", lambda: pamm.cache_append_fp8(c, x, x, n.long())),
        (ValueError, "new_len", lambda: pamm.cache_append_fp8(c, x, x, n, new_len=n[:1])),
        (ValueError, "on the GPU", lambda: pamm.cache_append_fp8(c, x, x, n)),
        (TypeError, "float8_e4m3fn", lambda: pamm.cache_append_fp8(c._replace(k=c.k.float()), x, x, n)),
        (TypeError, "float8_e4m3fn", lambda: pamm.attention_fp8(q, c._replace(v=c.v.view(torch.uint8)), n)),
        (ValueError, "share a shape", lambda: pamm.attention_fp8(q, c._replace(v=c.v[:, :64]), n)),
        (ValueError, "tails must hold", lambda: pamm.attention_fp8(q, c._replace(k_tail=c.k_tail[:, :7]), n)),
        (ValueError, "tails must have", lambda: pamm.attention_fp8(q, c._replace(v_tail=c.v_tail[:, :32]), n)),
        (TypeError, "tails must share", lambda: pamm.attention_fp8(q, c._replace(v_tail=c.v_tail.bfloat16()), n)),
        (ValueError, "k_scale must have", lambda: pamm.attention_fp8(q, c._replace(k_scale=c.k_scale[:, :1]), n)),
        (TypeError, "v_scale must be", lambda: pamm.attention_fp8(q, c._replace(v_scale=c.v_scale.double()), n)),
        (ValueError, "overlap itself", lambda: pamm.cache_append_fp8(
            c._replace(k_scale=c.k_scale[:, :, :1].expand(2, 2, 2)), x, x, n)),
        (ValueError, "does not fit", lambda: pamm.attention_fp8(q[:1], c, n)),
        (ValueError, "does not fit", lambda: pamm.attention_fp8(q[..., :16], c, n)),
        (ValueError, "share 2 key/value heads", lambda: pamm.attention_fp8(q[:, :, :3], c, n)),
        (TypeError, "share a dtype", lambda: pamm.attention_fp8(q.bfloat16(), c, n)),
        (ValueError, "kv_len", lambda: pamm.attention_fp8(q, c, n[:1])),
        (TypeError, "kv_len", lambda: pamm.attention_fp8(q, c, n.long())),
        (ValueError, "o must have", lambda: pamm.attention_fp8(q, c, n, o=q[:, :1])),
        (ValueError, "lse must be", lambda: pamm.attention_fp8(q, c, n, lse=torch.zeros(2, 3, 4))),
        (ValueError, "on the GPU", lambda: pamm.attention_fp8(q, c, n)),
    ]
    for kind, text, call in cases:
        with pytest.raises(kind, match=text):
            call()
