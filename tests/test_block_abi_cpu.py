"""Host-side checks of include/pamm_block.h (no GPU needed, no kernel
launched): exports, workspace sizes, and the refusal of invalid arguments
before anything is enqueued; the 64-bit definitions that the GPU tests use
against automatic differentiation and differences."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from activation_compression_pamm_amd import block_ops as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EUNSUP, EHIP, EVALUE, ETOOLARGE = range(10)
FAKE = 0x10000  # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pamm_block.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(pamm_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(ops._BLOCK_EXPORTS)
    for name in names:
        assert hasattr(lib, name)


def test_package_exports():
    for name in ("attention", "attention_backward", "add_rms_norm", "add_rms_norm_fp8", "add_rms_norm_backward",
                 "clip_grad_norm"):
        assert name in pamm.__all__ and callable(getattr(pamm, name))
    with pytest.raises(AttributeError):
        pamm.no_such_name


def problem(**kw):
    d = dict(dtype=1, causal=1, batch=2, seq_q=64, seq_k=64, heads=4, heads_kv=2, head_dim=64, window=0, scale=0.125,
             lse=FAKE)
    t = kw.pop("tensors", {})
    d.update(kw)
    p = ops._Attention(**d)
    for n in ("q", "k", "v", "o"):
        setattr(p, n, t.get(n, ops._Heads(FAKE, 64 * 4 * 64, 4 * 64, 64)))
    return p


def test_attention_validation(lib):
    def call(p, ws=None, n=0):
        return lib.pamm_attention(ctypes.byref(p), ws, n, None)

    assert lib.pamm_attention(None, None, 0, None) == ENULL
    assert call(problem(dtype=3)) == EDTYPE
    for kw in ({"batch": -1}, {"heads": 3}, {"heads_kv": 0}, {"heads": 0}, {"head_dim": 0}, {"head_dim": 136},
               {"seq_q": 2**31}, {"seq_k": -1}, {"seq_q": 2**31 - 1}, {"batch": 2**31 - 1}, {"heads": 2**62}):
        assert call(problem(**kw)) == ESHAPE, kw
    assert call(problem(head_dim=60)) == EALIGN
    for kw in ({"causal": 2}, {"scale": math.inf}, {"scale": math.nan}, {"window": -1}, {"window": 3, "causal": 0}):
        assert call(problem(**kw)) == EVALUE, kw
    assert call(problem(lse=None)) == ENULL
    assert call(problem(lse=FAKE + 2)) == EALIGN
    assert call(problem(kv_len=FAKE + 1)) == EALIGN
    for n in ("q", "k", "v", "o"):
        bad = {"data": None, "stride_b": 16384, "stride_s": 256, "stride_h": 64}
        assert call(problem(tensors={n: ops._Heads(**bad)})) == ENULL
        assert call(problem(tensors={n: ops._Heads(FAKE + 8, 16384, 256, 64)})) == EALIGN
        assert call(problem(tensors={n: ops._Heads(FAKE, 16384, 260, 64)})) == EALIGN
        assert call(problem(tensors={n: ops._Heads(FAKE, 16384, -256, 64)})) == ESHAPE
        assert call(problem(tensors={n: ops._Heads(FAKE, 2**41, 256, 64)})) == ESHAPE
        assert call(problem(tensors={n: ops._Heads(FAKE, 16384, 2**24, 64)})) == EUNSUP
    assert call(problem(batch=0)) == OK
    assert call(problem(seq_q=0)) == OK


def test_attention_workspace(lib):
    p = problem(seq_q=1, seq_k=8192)
    need = lib.pamm_attention_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert lib.pamm_attention(ctypes.byref(p), None, 0, None) == EWS
    assert lib.pamm_attention(ctypes.byref(p), FAKE, need - 1, None) == EWS
    assert lib.pamm_attention(ctypes.byref(p), FAKE + 16, need, None) == EALIGN
    p = problem(batch=64, seq_q=2048, seq_k=2048)
    assert lib.pamm_attention_workspace_size(ctypes.byref(p)) == 0
    assert lib.pamm_attention_backward_workspace_size(ctypes.byref(p)) >= 64 * 4 * 2048 * 4
    h = ops._Heads(FAKE, 16384, 256, 64)
    q = problem()
    r = ctypes.byref
    assert lib.pamm_attention_backward(r(q), None, r(h), r(h), r(h), FAKE, 1 << 20, None) == ENULL
    assert lib.pamm_attention_backward(r(q), r(h), r(h), r(h), r(h), None, 0, None) == EWS
    bad = ops._Heads(FAKE + 4, 16384, 256, 64)
    assert lib.pamm_attention_backward(r(q), r(h), r(h), r(bad), r(h), FAKE, 1 << 20, None) == EALIGN


def call_norm(lib, x=FAKE, ldx=64, r=None, ldr=64, w=FAKE, n=4, d=64, dt=1, eps=1e-6, h=None, ldh=64, y=FAKE, ldy=64,
              q=None, ldq=64, qs=None, rstd=FAKE):
    return lib.pamm_add_rms_norm(x, ldx, r, ldr, w, n, d, dt, eps, h, ldh, y, ldy, q, ldq, qs, rstd, None)


def test_norm_validation(lib):
    assert call_norm(lib, dt=9) == EDTYPE
    for kw in ({"n": -1}, {"d": 0}, {"d": 32776, "ldx": 40000}, {"ldx": 63}, {"ldy": 8}, {"n": 2**31},
               {"ldx": 2**41}, {"q": FAKE, "qs": FAKE, "ldq": 8}):
        assert call_norm(lib, **kw) == ESHAPE, kw
    for kw in ({"eps": -1.0}, {"eps": math.nan}, {"eps": math.inf}):
        assert call_norm(lib, **kw) == EVALUE
    for kw in ({"x": None}, {"w": None}, {"y": None}, {"r": FAKE}, {"q": FAKE}):
        assert call_norm(lib, **kw) == ENULL, kw
    for kw in ({"x": FAKE + 2}, {"ldx": 68}, {"w": FAKE + 8}, {"q": FAKE + 4, "qs": FAKE}, {"rstd": FAKE + 1},
               {"q": FAKE, "qs": FAKE, "ldq": 68}, {"r": FAKE, "h": FAKE + 4}):
        assert call_norm(lib, **kw) == EALIGN, kw
    assert call_norm(lib, n=0, x=None, w=None, y=None) == OK
    need = lib.pamm_add_rms_norm_backward_workspace_size(1000, 64, 1)
    assert need >= 64 * 4 and need % 256 == 0

    def back(dy=FAKE, h=FAKE, w=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, size=need, ld=64):
        return lib.pamm_add_rms_norm_backward(dy, ld, h, 64, w, rstd, None, 0, 1000, 64, 1, dx, 64, dw, ws, size, None)

    for kw in ({"dy": None}, {"h": None}, {"w": None}, {"rstd": None}, {"dx": None}, {"dw": None}):
        assert back(**kw) == ENULL, kw
    assert back(ws=None) == EWS and back(size=need - 1) == EWS and back(ws=FAKE + 8) == EALIGN
    assert back(ld=32) == ESHAPE and back(dy=FAKE + 4) == EALIGN


def test_clip_validation(lib):
    def call(grads, max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE, size=1 << 20, count=None):
        arr = (ops._Grad * max(1, len(grads)))(*[ops._Grad(*g) for g in grads])
        return lib.pamm_clip_grad_norm(arr, len(grads) if count is None else count, max_norm, eps, norm, ws, size, None)

    g = [FAKE, FAKE, 1, 100, 100, 100, 0, 0]

    def but(**kw):
        names = ["data", "out", "rows", "cols", "ld", "ld_out", "dtype", "out_dtype"]
        return [kw.get(n, x) for n, x in zip(names, g)]

    assert call([g], count=-1) == ESHAPE
    assert call([g], max_norm=-1.0) == EVALUE and call([g], max_norm=math.nan) == EVALUE
    assert call([g], eps=-1.0) == EVALUE and call([g], norm=None) == ENULL and call([g], norm=FAKE + 2) == EALIGN
    assert call([but(dtype=4)]) == EDTYPE and call([but(out_dtype=4)]) == EDTYPE
    assert call([but(data=None)]) == ENULL and call([but(out=None)]) == ENULL
    assert call([but(data=FAKE + 2, out=FAKE + 2)]) == EALIGN
    assert call([but(rows=-1)]) == ESHAPE and call([but(cols=2**41)]) == ESHAPE
    assert call([but(rows=5, ld=99)]) == ESHAPE
    assert call([but(out_dtype=1)]) == EVALUE  # in place with another type
    assert call([but(rows=2, ld_out=120)]) == EVALUE  # in place with other rows
    assert call([g], ws=None) == EWS and call([g], size=8) == EWS and call([g], ws=FAKE + 8) == EALIGN
    arr = (ops._Grad * 200)()
    assert lib.pamm_clip_grad_norm_workspace_size(arr, 200) > lib.pamm_clip_grad_norm_workspace_size(arr, 1) > 0


def test_definitions_against_automatic_differentiation():
    rng = np.random.default_rng(0)
    B, Sq, Sk, H, Hkv, D = 2, 19, 23, 4, 2, 8
    q, do = rng.standard_normal((B, Sq, H, D)), rng.standard_normal((B, Sq, H, D))
    k, v = rng.standard_normal((B, Sk, Hkv, D)), rng.standard_normal((B, Sk, Hkv, D))
    kw = {"causal": True, "window": 9, "q_len": [19, 12], "kv_len": [23, 9]}
    ref = bo.attention(q, k, v, do, **kw)
    t = [torch.from_numpy(x).requires_grad_(True) for x in (q, k, v)]
    o = torch.zeros(B, Sq, H, D, dtype=torch.float64)
    for b in range(B):
        m = torch.from_numpy(bo.visible(Sq, Sk, kw["q_len"][b], kw["kv_len"][b], True, 9))
        for h in range(H):
            s = (t[0][b, :, h] @ t[1][b, :, h // 2].T / math.sqrt(D)).masked_fill(~m, -1e300)
            p = torch.softmax(s, 1) * m.any(1)[:, None] * m
            o[b, :, h] = p @ t[2][b, :, h // 2]
    np.testing.assert_allclose(ref["o"], o.detach().numpy(), rtol=1e-12, atol=1e-14)
    for g, n in zip(torch.autograd.grad((o * torch.from_numpy(do)).sum(), t), ("dq", "dk", "dv")):
        np.testing.assert_allclose(ref[n], g.numpy(), rtol=1e-10, atol=1e-13)

    x, w, dy, dh = rng.standard_normal((5, 33)), rng.standard_normal(33), rng.standard_normal((5, 33)), rng.standard_normal((5, 33))
    x = x.astype(np.float32).astype(np.float64)
    ref = bo.add_rms_norm(x, w, dy=dy, dh=dh)
    a, b = torch.from_numpy(x).requires_grad_(True), torch.from_numpy(w).requires_grad_(True)
    y = a * torch.rsqrt((a * a).mean(1, keepdim=True) + 1e-6) * b
    np.testing.assert_allclose(ref["y"], y.detach().numpy(), rtol=1e-12)
    ga, gb = torch.autograd.grad((y * torch.from_numpy(dy)).sum(), (a, b))
    np.testing.assert_allclose(ref["dx"], ga.numpy() + dh, rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(ref["dw"], gb.numpy(), rtol=1e-10, atol=1e-13)


def test_e4m3_values():
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    table = np.unique(table[np.isfinite(table)])
    x = np.concatenate([table, (table[1:] + table[:-1]) / 2 * 1.0001, np.linspace(-500, 500, 777)])
    nearest = table[np.abs(np.clip(x, -448, 448)[:, None] - table[None]).argmin(1)]
    assert np.array_equal(bo.e4m3(x), nearest)


def test_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        pamm.attention(q, q, q)
    with pytest.raises(ValueError):
        pamm.add_rms_norm(torch.zeros(2, 8), torch.zeros(8))
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([torch.zeros(8)], 1.0)
