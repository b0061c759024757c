"""A transformer block's attention half around a PAMM projection.

"QKV Projections Require a Fraction of Their Memory", section 3 "Contributi
Chiave": the method is a plugin beside attention that keeps no probabilities.
Here both stand together with what surrounds them, each keeping little for
the backward pass:

    h = x + residual, y = norm(h)        keeps h, 1/rms of each row
    qkv = y W^T            (PammLinear)  keeps generators, index, scale
    o = softmax(q k^T) v                 keeps qkv, o, one number a row
    out = o W_o^T                        keeps o

and the gradients of all layers are clipped by their global norm.  For
serving, `PammAttentionBlock.step` takes new tokens (one or a chunk) over a
cache of keys and values, optionally with the norm's output in 8 bits.

    python -m activation_compression_pamm_amd.block [--steps 10] [--json]

trains one block for a few steps on synthetic clustered tokens, then decodes
with it and compares with the whole forward pass.
"""
from __future__ import annotations

import argparse
import json
import time

import torch
from torch.autograd.function import once_differentiable

from .autograd import PammLinear, _aligned_rows
from .block_ops import (add_rms_norm, add_rms_norm_backward, add_rms_norm_fp8, attention, attention_backward,
                        clip_grad_norm)

__all__ = ["AttentionFunction", "PackedAttentionFunction", "AddRMSNormFunction", "AddRMSNorm", "KVCache",
           "PammAttentionBlock", "differentiable_attention"]


def _aligned_heads(t):
    """t itself where its head rows are contiguous and start on 16 bytes, else
    a contiguous copy of its own (gradients arrive in any layout, also as
    contiguous views from anywhere in a buffer)."""
    size = t.element_size()
    if t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s * size % 16 == 0 for s in t.stride()[:-1]):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class AttentionFunction(torch.autograd.Function):
    """attention() with attention_backward() as its gradient; lse is returned
    too and carries no gradient."""

    @staticmethod
    def forward(ctx, q, k, v, causal, window, scale, q_len, kv_len):
        kw = {"causal": causal, "window": window, "scale": scale}
        o, lse = attention(q, k, v, q_len=q_len, kv_len=kv_len, **kw)
        ctx.save_for_backward(q, k, v, o, lse, q_len, kv_len)
        ctx.kw = kw
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, do, _):
        *saved, q_len, kv_len = ctx.saved_tensors
        dq, dk, dv = attention_backward(_aligned_heads(do), *saved, q_len=q_len, kv_len=kv_len, **ctx.kw)
        return dq, dk, dv, None, None, None, None, None


def differentiable_attention(q, k, v, *, causal=False, window=0, scale=None, q_len=None, kv_len=None):
    """attention() that autograd can go through; returns o alone."""
    return AttentionFunction.apply(q, k, v, causal, window, scale, q_len, kv_len)[0]


class PackedAttentionFunction(torch.autograd.Function):
    """Attention of the packed output of a projection, [B x S x (H + 2 Hkv) x D]:
    its gradient is written into one tensor of that layout, with no copies."""

    @staticmethod
    def forward(ctx, qkv, heads, heads_kv, causal, window, scale, lengths):
        kw = {"causal": causal, "window": window, "scale": scale}
        o, lse = attention(*qkv.split([heads, heads_kv, heads_kv], dim=2), q_len=lengths, kv_len=lengths, **kw)
        ctx.save_for_backward(qkv, o, lse, lengths)
        ctx.kw, ctx.sizes = kw, [heads, heads_kv, heads_kv]
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        qkv, o, lse, lengths = ctx.saved_tensors
        grad = torch.empty_like(qkv, memory_format=torch.contiguous_format)
        dq, dk, dv = grad.split(ctx.sizes, dim=2)
        attention_backward(_aligned_heads(do), *qkv.split(ctx.sizes, dim=2), o, lse, q_len=lengths, kv_len=lengths,
                           dq=dq, dk=dk, dv=dv, **ctx.kw)
        return grad, None, None, None, None, None, None


class AddRMSNormFunction(torch.autograd.Function):
    """(y, h) of add_rms_norm for x and residual [... x d]; only h, the weight
    and 1/rms are kept."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        d = x.shape[-1]
        x2 = _aligned_rows(x.reshape(-1, d))
        r2 = _aligned_rows(residual.reshape(-1, d)) if residual is not None else None
        y, h, rstd = add_rms_norm(x2, weight, r2, eps=eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.shape, ctx.has_residual = x.shape, residual is not None
        ctx.set_materialize_grads(False)
        if residual is None:
            return y.reshape(x.shape)
        return y.reshape(x.shape), h.reshape(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        d = h.shape[1]
        if dy is None:
            return dh, dh if ctx.has_residual else None, None, None
        dx, dw = add_rms_norm_backward(_aligned_rows(dy.reshape(-1, d)), h, weight, rstd,
                                       dh=_aligned_rows(dh.reshape(-1, d)) if dh is not None else None)
        dx = dx.reshape(ctx.shape)
        return dx, dx if ctx.has_residual else None, dw.to(weight.dtype), None


class AddRMSNorm(torch.nn.Module):
    """The residual addition and the root-mean-square norm after it: forward
    returns (y, h), h being the residual of what follows (x itself without
    one)."""

    def __init__(self, dim: int, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.eps = float(eps)

    def forward(self, x, residual=None):
        if residual is None:
            return AddRMSNormFunction.apply(x, None, self.weight, self.eps), x
        return AddRMSNormFunction.apply(x, residual, self.weight, self.eps)

    def extra_repr(self) -> str:
        return f"{self.weight.shape[0]}, eps={self.eps}"


class KVCache:
    """Keys and values [B x room x Hkv x D] of the tokens so far, lengths [B]
    int32 on the GPU."""

    def __init__(self, batch, room, heads_kv, head_dim, *, device="cuda", dtype=torch.bfloat16):
        self.k = torch.empty(batch, room, heads_kv, head_dim, device=device, dtype=dtype)
        self.v = torch.empty_like(self.k)
        self.lengths = torch.zeros(batch, device=device, dtype=torch.int32)
        self.used = 0  # the longest sequence, known on the host

    def append(self, k, v):
        """k, v [B x n x Hkv x D] behind each sequence's tokens."""
        batch, room, *head = self.k.shape
        if k.dim() != 4 or k.shape != v.shape or k.shape[0] != batch or list(k.shape[2:]) != head:
            raise ValueError(f"KVCache: k and v must be [{batch} x tokens x {head[0]} x {head[1]}], got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if k.dtype != self.k.dtype or v.dtype != self.v.dtype:
            raise TypeError(f"KVCache: k and v must be {self.k.dtype}, got {k.dtype} and {v.dtype}")
        n = k.shape[1]
        if self.used + n > room:
            raise ValueError(f"KVCache: {self.used} + {n} tokens do not fit {room}")
        at = self.lengths[:, None].long() + torch.arange(n, device=k.device)
        rows = torch.arange(batch, device=k.device)[:, None]
        self.k[rows, at] = k
        self.v[rows, at] = v
        self.lengths += n
        self.used += n


class PammAttentionBlock(torch.nn.Module):
    """Residual addition, norm, PammLinear for queries, keys and values, causal
    attention, output projection.

    forward(x, residual=None, lengths=None): x [B x S x dim] -> (out, h), to be
    given to the next block as x and residual; lengths [B] int32 are the valid
    tokens of each sequence."""

    def __init__(self, dim: int, heads: int, heads_kv: int | None = None, *, head_dim: int | None = None,
                 window: int = 0, ratio: int = 512, pamm_eps: float = 0.0, norm_eps: float = 1e-6, seed: int = 0,
                 device=None, dtype=None):
        super().__init__()
        self.heads, self.heads_kv = heads, heads_kv if heads_kv is not None else heads
        self.head_dim = head_dim if head_dim is not None else dim // heads
        self.window = int(window)
        self.norm = AddRMSNorm(dim, norm_eps, device=device, dtype=dtype)
        self.qkv = PammLinear(dim, (heads + 2 * self.heads_kv) * self.head_dim, bias=False, ratio=ratio, eps=pamm_eps,
                              seed=seed, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * self.head_dim, dim, bias=False, device=device, dtype=dtype)

    def _heads(self, qkv):
        return qkv.view(*qkv.shape[:2], self.heads + 2 * self.heads_kv, self.head_dim)

    def forward(self, x, residual=None, lengths=None):
        y, h = self.norm(x, residual)
        o = PackedAttentionFunction.apply(self._heads(self.qkv(y)), self.heads, self.heads_kv, True, self.window, None,
                                          lengths)
        return self.out(o.reshape(*x.shape[:2], -1)), h

    def cache(self, batch: int, room: int) -> KVCache:
        return KVCache(batch, room, self.heads_kv, self.head_dim, device=self.qkv.weight.device,
                       dtype=self.qkv.weight.dtype)

    def quantize_qkv(self):
        """The projection's weight as it is now in 8 bits, with a scale per
        output row: for step(eight_bits=...), as long as the weight stays."""
        w = self.qkv.weight.detach().float()
        scale = w.abs().amax(1).clamp(min=2.0 ** -100) / 448.0
        return (w / scale[:, None]).to(torch.float8_e4m3fn), scale[None, :]

    @torch.no_grad()
    def step(self, x, residual, cache: KVCache, *, eight_bits=False):
        """New tokens x [B x n x dim] over the cache: (out, h) as forward gives
        them for these tokens.  eight_bits: the norm's output and the
        projection in 8 bits, with the weight that quantize_qkv() gave; True
        lays out the present weight in every call, so the block keeps none
        that an update could leave behind."""
        d = x.shape[-1]
        if eight_bits:
            w8, w_scale = eight_bits if isinstance(eight_bits, tuple) else self.quantize_qkv()
            y8, y_scale, h, _ = add_rms_norm_fp8(_aligned_rows(x.reshape(-1, d)), self.norm.weight,
                                                 _aligned_rows(residual.reshape(-1, d)) if residual is not None else None,
                                                 eps=self.norm.eps)
            qkv = torch._scaled_mm(y8, w8.t(), scale_a=y_scale[:, None], scale_b=w_scale, out_dtype=torch.bfloat16)
            qkv, h = qkv.view(*x.shape[:2], -1).to(x.dtype), h.reshape(x.shape)
        else:
            y, h = self.norm(x, residual)
            qkv = torch.nn.functional.linear(y, self.qkv.weight)
        q, k, v = self._heads(qkv).split([self.heads, self.heads_kv, self.heads_kv], dim=2)
        cache.append(k, v)
        o, _ = attention(q, cache.k[:, :cache.used], cache.v[:, :cache.used], causal=True, window=self.window,
                         kv_len=cache.lengths)
        return self.out(o.reshape(*x.shape[:2], -1)), h


def run(steps: int = 10, batch: int = 4, seq: int = 1024, dim: int = 768, heads: int = 12, ratio: int = 64,
        decode: int = 32) -> dict:
    import numpy as np

    from . import synth

    torch.manual_seed(0)
    dev, dt = "cuda", torch.bfloat16
    block = PammAttentionBlock(dim, heads, ratio=ratio, seed=3, device=dev, dtype=dt)
    X = synth.clustered_activations(batch * seq, dim, 64, seed=5, dtype="bf16")
    X = torch.from_numpy(X.view(np.int16)).view(dt).to(dev).reshape(batch, seq, dim)
    target = torch.roll(X, 1, dims=1)  # each position is to give the token before it
    opt = torch.optim.SGD(block.parameters(), lr=8.0)
    losses, norms = [], []
    for i in range(steps + 1):
        if i == 1:  # the first step is not timed
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        opt.zero_grad(set_to_none=True)
        out, _ = block(X)
        loss = (out.float() - target.float()).square().mean()
        loss.backward()
        norms.append(clip_grad_norm([p.grad for p in block.parameters()], 1.0))
        opt.step()
        losses.append(loss.detach())
    torch.cuda.synchronize()
    train_s = (time.perf_counter() - t0) / steps

    block.eval()
    with torch.no_grad():
        whole, _ = block(X)
    cache = block.cache(batch, seq)
    start = seq - decode
    part, _ = block.step(X[:, :start], None, cache)
    got = [part]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(start, seq):
        got.append(block.step(X[:, i:i + 1], None, cache)[0])
    torch.cuda.synchronize()
    token_s = (time.perf_counter() - t0) / max(decode, 1)
    got = torch.cat(got, 1)
    off = float((got.float() - whole.float()).norm() / whole.float().norm())
    return {"losses": [round(float(x), 5) for x in losses], "gradient_norms": [round(float(x), 4) for x in norms],
            "ms_per_training_step": round(train_s * 1e3, 3), "us_per_token_step": round(token_s * 1e6, 1),
            "decode_against_forward": off}


def main():
    ap = argparse.ArgumentParser(description="Train and decode with one PAMM attention block.")
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--json", action="store_true")
    a = ap.parse_args()
    res = run(a.steps)
    if a.json:
        print(json.dumps(res))
    else:
        for k, v in res.items():
            print(f"{k}: {v}")


if __name__ == "__main__":
    main()
