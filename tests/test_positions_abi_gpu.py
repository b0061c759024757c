"""GPU: what include/pamm_positions.h allows and the binding does not ask for:
the rotation of queries and keys in one call without a norm, and the norm,
with its gradients, where there are no keys."""
import ctypes

import numpy as np
import pytest
import torch

import position_oracle as po
from activation_compression_pamm_amd import position_ops as ops
from activation_compression_pamm_amd.block_ops import _Heads
from test_attention_gpu import close, dev, host, say, values
from test_positions_cpu import Rotary
from test_positions_gpu import BOTH, KINDS, freqs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def heads(t):
    return _Heads(t.data_ptr(), *t.stride()[:3])


def call(name, p, *args):
    stream = torch.cuda.current_stream().cuda_stream
    assert getattr(ops._lib(), name)(ctypes.byref(p), *args, stream) == 0
    torch.cuda.synchronize()


def problem(dtype, f, interleaved, q, qo, k=None, ko=None, **kw):
    B, S, H, D = q.shape
    p = Rotary(dtype=0 if dtype == "f32" else 1, interleaved=int(interleaved), batch=B, seq=S, heads_q=H, head_dim=D,
               rot_dim=2 * len(f), magnitude=1.0, eps=1e-6, inv_freq=f.data_ptr(), q=heads(q), q_out=heads(qo), **kw)
    if k is not None:
        p.heads_k, p.k, p.k_out = k.shape[2], heads(k), heads(ko)
    return p


@BOTH
@KINDS
@pytest.mark.parametrize("B,S,H,Hkv", [(1, 1, 4, 4), (3, 77, 8, 2), (2, 700, 2, 6), (4, 1025, 12, 1)])
@pytest.mark.parametrize("D,rot", [(64, 64), (40, 20), (128, 32)])
def test_queries_and_keys_without_a_norm(dtype, interleaved, B, S, H, Hkv, D, rot):
    say("rotation of two tensors", dtype, interleaved, B, S, H, Hkv, D, rot)
    rng = np.random.default_rng(0)
    x = [values(rng, (B, S, h, D), dtype) for h in (H, Hkv)]
    q, k = (dev(t, dtype) for t in x)
    f, out = freqs(rot), [torch.full_like(t, 9.0) for t in (q, k)]
    for inverse in (0, 1):
        call("pamm_rotary", problem(dtype, f, interleaved, q, out[0], k, out[1], inverse=inverse))
        for t, got in zip(x, out):
            y, tol = po.rotary(t, np.broadcast_to(np.arange(S), (B, S)), host(f), dtype=dtype, interleaved=interleaved,
                               inverse=bool(inverse))
            close("rotary", got, y, tol)


@BOTH
@pytest.mark.parametrize("B,S,H,D,rot", [(1, 1, 4, 64, 64), (3, 333, 5, 72, 18), (2, 1000, 8, 128, 64)])
def test_a_norm_without_keys(dtype, B, S, H, D, rot):
    say("norm of one tensor", dtype, B, S, H, D, rot)
    rng = np.random.default_rng(1)
    x, dy, w = values(rng, (B, S, H, D), dtype), values(rng, (B, S, H, D), dtype), host(dev(1 + 0.2 * rng.standard_normal(D), dtype))
    q, g, wd, f = dev(x, dtype), dev(dy, dtype), dev(w, dtype), freqs(rot)
    y, dx, dw = torch.full_like(q, 9.0), torch.full_like(q, 9.0), torch.full((D,), 9.0, device="cuda")
    call("pamm_rotary", problem(dtype, f, False, q, y, q_weight=wd.data_ptr()))
    p = problem(dtype, f, False, q, dx, q_weight=wd.data_ptr())
    need = ops._lib().pamm_rotary_backward_workspace_size(ctypes.byref(p))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call("pamm_rotary_backward", p, ctypes.byref(heads(g)), None, dw.data_ptr(), None, ws.data_ptr(), need)
    ref = po.norm_rotary(x, w, np.broadcast_to(np.arange(S), (B, S)), host(f), dy=dy, dtype=dtype)
    for n, t in (("y", y), ("dx", dx), ("dw", dw)):
        close(n, t, ref[n], ref[n + "_tol"])
