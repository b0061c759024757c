"""A transformer block's attention half around a PAMM projection.

"QKV Projections Require a Fraction of Their Memory", section 3 "Contributi
Chiave": the method is a plugin beside attention that keeps no probabilities.
Here both stand together with what surrounds them, each keeping little for
the backward pass:

    h = x + residual, y = norm(h)        keeps h, 1/rms of each row
    qkv = y W^T            (PammLinear)  keeps generators, index, scale
    o = softmax(q k^T) v                 keeps qkv, o, one number a row
    out = o W_o^T                        keeps o

and the gradients of all layers are clipped by their global norm.  Queries and
keys may be normed for each head and rotated by their positions on the way;
that is done again in the backward pass from the kept qkv, so it keeps nothing.
For serving, `PammAttentionBlock.step` takes new tokens (one or a chunk) over a
cache of keys and values, optionally held in 8 bits, and optionally with the
norm's output in 8 bits.

    python -m activation_compression_pamm_amd.block [--steps 10] [--rotary] [--qk-norm] [--cache8] [--json]

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
from .cache_ops import CacheFP8, attention_fp8, cache_append_fp8
from .position_ops import qk_norm_rotary, qk_norm_rotary_backward, rotary, rotary_frequencies

__all__ = ["AttentionFunction", "PackedAttentionFunction", "PositionedAttentionFunction", "AddRMSNormFunction",
           "AddRMSNorm", "KVCache", "KVCache8", "PammAttentionBlock", "differentiable_attention"]


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


class PositionedAttentionFunction(torch.autograd.Function):
    """PackedAttentionFunction with queries and keys normed for each head and
    rotated by their positions.  Only qkv, o and lse are kept: what goes into
    the products is formed again in the backward pass."""

    @staticmethod
    def _turned(qkv, q_weight, k_weight, inv_freq, sizes, kw, eps):
        """Queries and keys as the products take them, side by side."""
        H, K, _ = sizes
        if q_weight is None:  # one call for both
            return rotary(qkv[:, :, :H + K], inv_freq, **kw).split([H, K], dim=2)
        both = torch.empty((*qkv.shape[:2], H + K, qkv.shape[3]), dtype=qkv.dtype, device=qkv.device)
        q, k, _ = qkv.split(sizes, dim=2)
        qo, ko = both.split([H, K], dim=2)
        return qk_norm_rotary(q, k, q_weight, k_weight, inv_freq, eps=eps, q_out=qo, k_out=ko, **kw)

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, inv_freq, positions, heads, heads_kv, causal, window, scale, lengths,
                interleaved, magnitude, eps):
        ctx.sizes, ctx.eps = [heads, heads_kv, heads_kv], eps
        ctx.kw = {"causal": causal, "window": window, "scale": scale}
        ctx.turn = {"interleaved": interleaved, "magnitude": magnitude}
        q, k = PositionedAttentionFunction._turned(qkv, q_weight, k_weight, inv_freq, ctx.sizes,
                                                   dict(ctx.turn, positions=positions), eps)
        o, lse = attention(q, k, qkv[:, :, heads + heads_kv:], q_len=lengths, kv_len=lengths, **ctx.kw)
        ctx.save_for_backward(qkv, q_weight, k_weight, inv_freq, positions, o, lse, lengths)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        qkv, q_weight, k_weight, inv_freq, positions, o, lse, lengths = ctx.saved_tensors
        turn = dict(ctx.turn, positions=positions)
        q, k = PositionedAttentionFunction._turned(qkv, q_weight, k_weight, inv_freq, ctx.sizes, turn, ctx.eps)
        grad = torch.empty_like(qkv, memory_format=torch.contiguous_format)
        dq, dk, dv = grad.split(ctx.sizes, dim=2)
        attention_backward(_aligned_heads(do), q, k, qkv[:, :, ctx.sizes[0] + ctx.sizes[1]:], o, lse, q_len=lengths,
                           kv_len=lengths, dq=dq, dk=dk, dv=dv, **ctx.kw)
        dwq = dwk = None
        if q_weight is not None:
            q, k, _ = qkv.split(ctx.sizes, dim=2)
            _, _, dwq, dwk = qk_norm_rotary_backward(dq, dk, q, k, q_weight, k_weight, inv_freq, eps=ctx.eps, dq_out=dq,
                                                     dk_out=dk, **turn)
            dwq, dwk = dwq.to(q_weight.dtype), dwk.to(k_weight.dtype)
        else:
            both = grad[:, :, :ctx.sizes[0] + ctx.sizes[1]]
            rotary(both, inv_freq, inverse=True, out=both, **turn)
        return (grad, dwq, dwk, *([None] * 11))


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


class _Lengths:
    """Of a cache: lengths [B] int32 on the GPU, and used, the longest of them,
    on the host.  Replays of a captured call move lengths alone.  So a call
    attends over the whole room while it is captured, and from then on one
    that is not captured asks the GPU for used, and waits for it."""

    def _begin(self, batch, device):
        self.lengths = torch.zeros(batch, device=device, dtype=torch.int32)
        self.used = 0
        self._replayed = False

    def _captured(self):
        """Whether this call is being captured; if not, used is up to date."""
        if self.lengths.is_cuda and torch.cuda.is_current_stream_capturing():
            self._replayed = True
            return True
        if self._replayed:
            self.used = max(self.lengths.tolist(), default=0)
        return False


class KVCache(_Lengths):
    """Keys and values [B x room x Hkv x D] of the tokens so far.  Tokens that
    replays of a captured call bring past the room are dropped."""

    def __init__(self, batch, room, heads_kv, head_dim, *, device="cuda", dtype=torch.bfloat16):
        self.k = torch.empty(batch, room, heads_kv, head_dim, device=device, dtype=dtype)
        self.v = torch.empty_like(self.k)
        self._begin(batch, device)

    def append(self, k, v):
        """k, v [B x n x Hkv x D] behind each sequence's tokens."""
        batch, room, *head = self.k.shape
        if k.dim() != 4 or k.shape != v.shape or k.shape[0] != batch or list(k.shape[2:]) != head:
            raise ValueError(f"KVCache: k and v must be [{batch} x tokens x {head[0]} x {head[1]}], got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if k.dtype != self.k.dtype or v.dtype != self.v.dtype:
            raise TypeError(f"KVCache: k and v must be {self.k.dtype}, got {k.dtype} and {v.dtype}")
        n, captured = k.shape[1], self._captured()
        if self.used + n > room:
            raise ValueError(f"KVCache: {self.used} + {n} tokens do not fit {room}")
        if n == 0:
            return
        new, rows = torch.arange(n, device=k.device), torch.arange(batch, device=k.device)[:, None]
        at = self.lengths[:, None].long() + new
        if captured:  # replays know of no limit: what does not fit repeats the last write that does, or changes nothing
            last = (room - 1 - self.lengths[:, None].long()).clamp(min=0)
            at, new = at.clamp(max=room - 1), torch.minimum(new, last)
            full = (self.lengths >= room)[:, None, None, None]
            k, v = (torch.where(full, old[rows, at], x[rows, new]) for old, x in ((self.k, k), (self.v, v)))
        self.k[rows, at] = k
        self.v[rows, at] = v
        if captured:
            self.lengths.add_(n).clamp_(max=room)
        else:
            self.lengths += n
            self.used += n

    def attend(self, q, window=0):
        """Causal attention of the newest tokens' queries [B x n x H x D]."""
        rows = self.k.shape[1] if self._captured() else self.used
        return attention(q, self.k[:, :rows], self.v[:, :rows], causal=True, window=window, kv_len=self.lengths)[0]


class KVCache8(_Lengths):
    """KVCache in 8 bits, with a scale for each block of tokens and head: half
    of bf16's memory, and of what a new token's attention has to read.  Tokens
    of the last, partial block stay in dtype until it is whole.  Tokens that
    replays of a captured call bring past the room are dropped."""

    def __init__(self, batch, room, heads_kv, head_dim, *, block=64, device="cuda", dtype=torch.bfloat16):
        self.tensors = CacheFP8.empty(batch, room, heads_kv, head_dim, block=block, device=device, dtype=dtype)
        self._begin(batch, device)

    def append(self, k, v):
        """k, v [B x n x Hkv x D] behind each sequence's tokens."""
        room, captured = self.tensors.k.shape[1], self._captured()
        if k.dim() == 4 and self.used + k.shape[1] > room:
            raise ValueError(f"KVCache8: {self.used} + {k.shape[1]} tokens do not fit {room}")
        cache_append_fp8(self.tensors, k, v, self.lengths)
        if not captured:
            self.used += k.shape[1]

    def attend(self, q, window=0):
        """Causal attention of the newest tokens' queries [B x n x H x D]."""
        c = self.tensors
        rows = c.k.shape[1] if self._captured() else self.used
        return attention_fp8(q, c._replace(k=c.k[:, :rows], v=c.v[:, :rows]), self.lengths, causal=True, window=window)[0]


class PammAttentionBlock(torch.nn.Module):
    """Residual addition, norm, PammLinear for queries, keys and values, causal
    attention, output projection.

    forward(x, residual=None, lengths=None, positions=None): x [B x S x dim] ->
    (out, h), to be given to the next block as x and residual; lengths [B] int32
    are the valid tokens of each sequence, positions [B x S] or [S] int64 or
    int32 those of the rotation (0, 1, ... by default).

    rotary: how many elements of each query and key head are rotated by their
    position (True: all), with rotary_base, rotary_interleaved and
    rotary_scaling (arguments of rotary_frequencies: scaling, factor, ...).
    qk_norm: queries and keys are normed for each head before that."""

    def __init__(self, dim: int, heads: int, heads_kv: int | None = None, *, head_dim: int | None = None,
                 window: int = 0, ratio: int = 512, pamm_eps: float = 0.0, norm_eps: float = 1e-6, seed: int = 0,
                 rotary: int | bool = 0, rotary_base: float = 10000.0, rotary_interleaved: bool = False,
                 rotary_scaling: dict | None = None, qk_norm: bool = False, device=None, dtype=None):
        super().__init__()
        self.heads, self.heads_kv = heads, heads_kv if heads_kv is not None else heads
        self.head_dim = head_dim if head_dim is not None else dim // heads
        self.window = int(window)
        self.norm = AddRMSNorm(dim, norm_eps, device=device, dtype=dtype)
        self.qkv = PammLinear(dim, (heads + 2 * self.heads_kv) * self.head_dim, bias=False, ratio=ratio, eps=pamm_eps,
                              seed=seed, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * self.head_dim, dim, bias=False, device=device, dtype=dtype)
        self.q_norm = self.k_norm = None
        if qk_norm:
            self.q_norm, self.k_norm = (torch.nn.Parameter(torch.ones(self.head_dim, device=device, dtype=dtype))
                                        for _ in range(2))
        self.interleaved = bool(rotary_interleaved)
        self.rotary_dim = self.head_dim if rotary is True else int(rotary)
        if not 0 <= self.rotary_dim <= self.head_dim:
            raise ValueError(f"PammAttentionBlock: rotary must be at most the head dimension {self.head_dim}, got {rotary}")
        # 64 bits, whatever the module is cast to: no buffer
        self._inv_freq, self.magnitude = None, 1.0
        if self.rotary_dim:
            self._inv_freq, self.magnitude = rotary_frequencies(self.rotary_dim, rotary_base, device="cpu",
                                                                **(rotary_scaling or {}))

    def _heads(self, qkv):
        return qkv.view(*qkv.shape[:2], self.heads + 2 * self.heads_kv, self.head_dim)

    def _frequencies(self, device):
        if self._inv_freq is not None and self._inv_freq.device != device:
            self._inv_freq = self._inv_freq.to(device)
        return self._inv_freq

    def forward(self, x, residual=None, lengths=None, positions=None):
        if positions is not None and not self.rotary_dim:
            raise ValueError("PammAttentionBlock: positions are given, but the block has no rotary positions")
        y, h = self.norm(x, residual)
        qkv = self._heads(self.qkv(y))
        if self.rotary_dim or self.q_norm is not None:
            o = PositionedAttentionFunction.apply(qkv, self.q_norm, self.k_norm, self._frequencies(x.device), positions,
                                                  self.heads, self.heads_kv, True, self.window, None, lengths,
                                                  self.interleaved, self.magnitude, self.norm.eps)
        else:
            o = PackedAttentionFunction.apply(qkv, self.heads, self.heads_kv, True, self.window, None, lengths)
        return self.out(o.reshape(*x.shape[:2], -1)), h

    def cache(self, batch: int, room: int, *, eight_bits: bool = False, block: int = 64):
        """An empty cache for step(): keys and values in the block's type, or
        with eight_bits in 8 bits, `block` tokens to a scale."""
        kw = {"device": self.qkv.weight.device, "dtype": self.qkv.weight.dtype}
        if eight_bits:
            return KVCache8(batch, room, self.heads_kv, self.head_dim, block=block, **kw)
        return KVCache(batch, room, self.heads_kv, self.head_dim, **kw)

    def quantize_qkv(self):
        """The projection's weight as it is now in 8 bits, with a scale per
        output row: for step(eight_bits=...), as long as the weight stays."""
        w = self.qkv.weight.detach().float()
        scale = w.abs().amax(1).clamp(min=2.0 ** -100) / 448.0
        return (w / scale[:, None]).to(torch.float8_e4m3fn), scale[None, :]

    @torch.no_grad()
    def step(self, x, residual, cache: KVCache | KVCache8, *, eight_bits=False):
        """New tokens x [B x n x dim] over the cache: (out, h) as forward gives
        them for these tokens, whose positions follow those in the cache.  eight_bits: the norm's output and the
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
        qkv = self._heads(qkv)
        q, k, v = qkv.split([self.heads, self.heads_kv, self.heads_kv], dim=2)
        if self.rotary_dim or self.q_norm is not None:  # in place: the projection's output is this call's own
            kw = {"offset": cache.lengths, "interleaved": self.interleaved, "magnitude": self.magnitude}
            freq = self._frequencies(x.device)
            if self.q_norm is not None:
                qk_norm_rotary(q, k, self.q_norm, self.k_norm, freq, eps=self.norm.eps, q_out=q, k_out=k, **kw)
            else:
                both = qkv[:, :, :self.heads + self.heads_kv]
                rotary(both, freq, out=both, **kw)
        cache.append(k, v)
        o = cache.attend(q, self.window)
        return self.out(o.reshape(*x.shape[:2], -1)), h


def run(steps: int = 10, batch: int = 4, seq: int = 1024, dim: int = 768, heads: int = 12, ratio: int = 64,
        decode: int = 32, rotary: bool = False, qk_norm: bool = False, cache8: bool = False) -> dict:
    import numpy as np

    from . import synth

    torch.manual_seed(0)
    dev, dt = "cuda", torch.bfloat16
    block = PammAttentionBlock(dim, heads, ratio=ratio, seed=3, rotary=rotary, qk_norm=qk_norm, device=dev, dtype=dt)
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
    cache = block.cache(batch, seq, eight_bits=cache8)
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
    ap.add_argument("--rotary", action="store_true", help="rotary positions")
    ap.add_argument("--qk-norm", action="store_true", help="norms of queries and keys for each head")
    ap.add_argument("--cache8", action="store_true", help="decode over a cache in 8 bits")
    ap.add_argument("--json", action="store_true")
    a = ap.parse_args()
    res = run(a.steps, rotary=a.rotary, qk_norm=a.qk_norm, cache8=a.cache8)
    if a.json:
        print(json.dumps(res))
    else:
        for k, v in res.items():
            print(f"{k}: {v}")


if __name__ == "__main__":
    main()
