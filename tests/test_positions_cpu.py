"""Host-side checks of include/pamm_positions.h and its binding (no GPU needed,
no kernel launched): exports, refusals, workspace sizes, the frequencies, and
the 64-bit definitions that the GPU tests use against automatic
differentiation."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import position_oracle as po
from activation_compression_pamm_amd import position_ops as ops
from activation_compression_pamm_amd.block_ops import _Heads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EUNSUP, EHIP, EVALUE, ETOOLARGE = range(10)
FAKE = 0x10000  # an aligned, never-dereferenced address


class Rotary(ctypes.Structure):
    """pamm_rotary_t"""
    _i, _l, _f, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    _fields_ = [("dtype", _i), ("interleaved", _i), ("inverse", _i), ("positions_64", _i), ("batch", _l), ("seq", _l),
                ("heads_q", _l), ("heads_k", _l), ("head_dim", _l), ("rot_dim", _l), ("magnitude", _f), ("eps", _f),
                ("inv_freq", _p), ("positions", _p), ("position_stride_b", _l), ("position_stride_s", _l),
                ("offset", _p), ("q_weight", _p), ("k_weight", _p), ("q", _Heads), ("k", _Heads), ("q_out", _Heads),
                ("k_out", _Heads)]


def problem(**kw):
    d = dict(dtype=1, batch=2, seq=5, heads_q=4, heads_k=2, head_dim=64, rot_dim=64, magnitude=1.0, eps=1e-6,
             inv_freq=FAKE, q_weight=FAKE, k_weight=FAKE)
    d.update(kw)
    p = Rotary(**d)
    for n in ("q", "k", "q_out", "k_out"):
        if n not in kw:
            setattr(p, n, _Heads(FAKE, 5 * 4 * 64, 4 * 64, 64))
    return p


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pamm_positions.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(pamm_[a-z_0-9]+)\s*\(", text))) == sorted(ops._POSITION_EXPORTS)
    for name in ops._POSITION_EXPORTS:
        assert hasattr(lib, name)
    for name in ops.__all__:
        assert name in pamm.__all__ and callable(getattr(pamm, name))


def test_the_packed_struct_is_the_declared_one():
    assert ctypes.sizeof(Rotary) == len(ops._pack_rotary(*range(10), 1.0, 2.0, *range(12, 35)))
    p = Rotary.from_buffer_copy(ops._pack_rotary(*range(10), 1.5, 2.5, *range(12, 35)))
    assert (p.positions_64, p.batch, p.rot_dim, p.magnitude, p.eps, p.inv_freq, p.positions) == (3, 4, 9, 1.5, 2.5, 12, 13)
    assert (p.position_stride_s, p.offset, p.q_weight, p.k_weight, p.q.data, p.k_out.stride_h) == (15, 16, 17, 18, 19, 34)


H = lambda *a: _Heads(*a)
BAD = [
    (dict(dtype=2), EDTYPE), (dict(batch=-1), ESHAPE), (dict(seq=-1), ESHAPE), (dict(batch=1 << 20, seq=1 << 20), ESHAPE),
    (dict(batch=1 << 62, seq=1 << 62), ESHAPE), (dict(heads_q=0), ESHAPE), (dict(heads_k=-1), ESHAPE),
    (dict(heads_q=1 << 40), ESHAPE), (dict(head_dim=0), ESHAPE), (dict(head_dim=136), ESHAPE), (dict(head_dim=60, rot_dim=60), EALIGN),
    (dict(rot_dim=-2), ESHAPE), (dict(rot_dim=7), ESHAPE), (dict(rot_dim=66), ESHAPE), (dict(interleaved=2), EVALUE),
    (dict(inverse=-1), EVALUE), (dict(positions_64=3), EVALUE), (dict(inverse=1), EVALUE),
    (dict(magnitude=math.inf), EVALUE), (dict(magnitude=math.nan), EVALUE), (dict(eps=-1e-6), EVALUE),
    (dict(eps=math.nan), EVALUE), (dict(eps=math.inf), EVALUE), (dict(inv_freq=None), ENULL), (dict(inv_freq=FAKE + 4), EALIGN),
    (dict(q_weight=None), ENULL), (dict(k_weight=None), ENULL), (dict(q_weight=FAKE + 8), EALIGN), (dict(heads_k=0), ENULL),
    (dict(positions=FAKE + 4, positions_64=1), EALIGN), (dict(positions=FAKE + 2), EALIGN),
    (dict(positions=FAKE, position_stride_b=-1), ESHAPE), (dict(positions=FAKE, position_stride_s=1 << 50), ESHAPE),
    (dict(offset=FAKE + 2), EALIGN), (dict(q=H(None, 1280, 256, 64)), ENULL), (dict(k=H(FAKE + 2, 1280, 256, 64)), EALIGN),
    (dict(q_out=H(FAKE, 1280, 256, 63)), EALIGN), (dict(k_out=H(FAKE, -8, 256, 64)), ESHAPE),
    (dict(q=H(FAKE, 1 << 45, 256, 64)), ESHAPE),
]


@pytest.mark.parametrize("kw,status", BAD, ids=[str(i) for i in range(len(BAD))])
def test_refusals(lib, kw, status):
    p = problem(**kw)
    assert lib.pamm_rotary(ctypes.byref(p), None) == status
    h = ctypes.byref(_Heads(FAKE, 1280, 256, 64))
    assert lib.pamm_rotary_backward(ctypes.byref(p), h, h, FAKE, FAKE, FAKE, 1 << 30, None) == status


def test_refusals_of_the_backward_pass(lib):
    h = ctypes.byref(_Heads(FAKE, 1280, 256, 64))
    p = ctypes.byref(problem())
    need = lib.pamm_rotary_backward_workspace_size(p)
    assert need > 0 and need % 256 == 0

    def call(p=p, dq=h, dk=h, dwq=FAKE, dwk=FAKE, ws=FAKE, n=need):
        return lib.pamm_rotary_backward(p, dq, dk, dwq, dwk, ws, n, None)

    assert lib.pamm_rotary(None, None) == ENULL and call(p=None) == ENULL
    assert lib.pamm_rotary_backward_workspace_size(None) == 0
    assert call(dq=None) == ENULL and call(dk=None) == ENULL and call(dwq=None) == ENULL and call(dwk=None) == ENULL
    assert call(dwq=FAKE + 2) == EALIGN and call(ws=None) == EWS and call(n=need - 1) == EWS and call(ws=FAKE + 16) == EALIGN
    assert call(p=ctypes.byref(problem(q_weight=None, k_weight=None))) == ENULL
    assert call(dq=ctypes.byref(_Heads(FAKE + 4, 1280, 256, 64))) == EALIGN
    # nothing to do is no error, and no launch
    for kw in (dict(batch=0), dict(seq=0)):
        assert lib.pamm_rotary(ctypes.byref(problem(**kw)), None) == OK


def test_arguments_are_checked_before_the_gpu_is_asked():
    f = torch.ones(8, dtype=torch.float64)
    x, w = torch.zeros(2, 3, 4, 16), torch.ones(16)
    cases = [
        (ValueError, "4-D", lambda: pamm.rotary(x[0], f)),
        (ValueError, "stride 1", lambda: pamm.rotary(x.transpose(2, 3), f)),
        (TypeError, "float64", lambda: pamm.rotary(x, f.float())),
        (ValueError, "do not fit", lambda: pamm.rotary(x, torch.ones(9, dtype=torch.float64))),
        (ValueError, "inv_freq", lambda: pamm.rotary(x, None)),
        (ValueError, "1-D", lambda: pamm.rotary(x, f[None])),
        (ValueError, "positions must have shape", lambda: pamm.rotary(x, f, positions=torch.zeros(4, dtype=torch.int64))),
        (TypeError, "int64 or int32", lambda: pamm.rotary(x, f, positions=torch.zeros(3))),
        (ValueError, "offset", lambda: pamm.rotary(x, f, offset=torch.zeros(3, dtype=torch.int32))),
        (TypeError, "int32", lambda: pamm.rotary(x, f, offset=torch.zeros(2, dtype=torch.int64))),
        (ValueError, "out must be", lambda: pamm.rotary(x, f, out=x[:1])),
        (ValueError, "overlap itself", lambda: pamm.rotary(x, f, out=x[:1].expand(2, 3, 4, 16))),
        (TypeError, "float32 and bfloat16", lambda: pamm.rotary(x.half(), f)),
        (ValueError, "on the GPU", lambda: pamm.rotary(x, f)),
        (ValueError, "k must be", lambda: pamm.qk_norm_rotary(x, x[:, :2], w, w, f)),
        (TypeError, "share a dtype", lambda: pamm.qk_norm_rotary(x, x.bfloat16(), w, w, f)),
        (ValueError, "are needed", lambda: pamm.qk_norm_rotary(x, x, w, None, f)),
        (ValueError, "k_weight", lambda: pamm.qk_norm_rotary(x, x, w, w[:8], f)),
        (ValueError, "k_weight", lambda: pamm.qk_norm_rotary(x, x, w, w.bfloat16(), f)),
        (ValueError, "dk must be", lambda: pamm.qk_norm_rotary_backward(x, x[:1], x, x, w, w, f)),
        (ValueError, "on the GPU", lambda: pamm.qk_norm_rotary_backward(x, x, x, x, w, w, f)),
    ]
    for kind, text, call in cases:
        with pytest.raises(kind, match=text):
            call()


def test_frequencies():
    def of(dim, *a, **kw):
        return pamm.rotary_frequencies(dim, *a, device="cpu", **kw)

    f, m = of(64)
    assert f.dtype == torch.float64 and m == 1.0
    assert all(abs(float(f[j]) - 10000.0 ** (-j / 32)) <= 1e-15 for j in range(32))
    assert torch.equal(of(64, scaling="linear", factor=4)[0], f / 4)
    g, m = of(64, scaling="ntk", factor=4)
    assert m == 1.0 and float(g[0]) == 1.0 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12
    g, m = of(64, scaling="yarn", factor=4, original_length=4096)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-15
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(g[turns >= 40], f[turns >= 40]) and torch.allclose(g[turns <= 0.7], f[turns <= 0.7] / 4, rtol=1e-15)
    assert (g <= f).all() and (g >= f / 4 * (1 - 1e-15)).all() and (g[1:] < g[:-1]).all()
    assert of(0)[0].shape == (0,) and of(2, scaling="ntk", factor=2)[0].tolist() == [1.0]
    for kw in (dict(dim=7), dict(dim=-2), dict(dim=8, base=0.0), dict(dim=8, factor=0.5, scaling="linear"),
               dict(dim=8, factor=2.0), dict(dim=8, scaling="other"), dict(dim=8, scaling="yarn", factor=2.0),
               dict(dim=8, scaling="yarn", factor=2.0, original_length=100, turns=(4, 2)), dict(dim=8, base=math.nan)):
        with pytest.raises(ValueError, match="rotary_frequencies"):
            of(**kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 6, 16])
def test_oracle_against_automatic_differentiation(interleaved, rot):
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((2, 3, 4, 16)), rng.standard_normal((2, 3, 4, 16)), rng.standard_normal(16)
    pos, f, kw = rng.integers(0, 99, (2, 3)), rng.random(rot // 2), dict(interleaved=interleaved, magnitude=1.3)
    ref = po.norm_rotary(x, w, pos, f, eps=0.1, dy=dy, **kw)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = tx / torch.sqrt((tx * tx).mean(-1, keepdim=True) + 0.1) * tw
    t = torch.tensor(po.angles(pos, f))
    a, b = po.split(n, rot, interleaved)
    ya, yb = 1.3 * (a * t.cos() - b * t.sin()), 1.3 * (a * t.sin() + b * t.cos())
    y = torch.cat([torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1), n[..., rot:]], -1)
    gx, gw = torch.autograd.grad(y, (tx, tw), torch.tensor(dy))
    assert np.allclose(ref["y"], y.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(ref["dx"], gx.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(ref["dw"], gw.numpy(), rtol=1e-11, atol=1e-13)
