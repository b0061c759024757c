"""GPU: the attention block (norm, PammLinear, attention, output projection)
against a plain 64-bit one, its decoding against its forward pass, and the
autograd wrappers of the operators."""
import math

import pytest
import torch

import activation_compression_pamm_amd as pamm
from activation_compression_pamm_amd.block import (AddRMSNorm, KVCache, PammAttentionBlock, differentiable_attention,
                                                   run)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def plain_block(block, x, residual, lengths=None):
    """The block's definition on CPU in 64 bits, with gradients by autograd."""
    p = {n: t.detach().double().cpu().requires_grad_(True) for n, t in block.named_parameters()}
    x, residual = x.detach().double().cpu().requires_grad_(True), residual.detach().double().cpu().requires_grad_(True)
    h = x + residual
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + block.norm.eps) * p["norm.weight"]
    B, S, _ = x.shape
    H, K, D = block.heads, block.heads_kv, block.head_dim
    q, k, v = (y @ p["qkv.weight"].T).view(B, S, H + 2 * K, D).split([H, K, K], dim=2)
    k, v = k.repeat_interleave(H // K, 2), v.repeat_interleave(H // K, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    i, j = torch.arange(S)[:, None], torch.arange(S)[None]
    m = j <= i
    if block.window:
        m = m & (j > i - block.window)
    m = m[None].repeat(B, 1, 1)
    if lengths is not None:
        m = m & (torch.arange(S)[None, :, None] < lengths[:, None, None]) & (j[None] < lengths[:, None, None])
    s = s.masked_fill(~m[:, None], -1e300)
    a = torch.softmax(s, -1) * m[:, None]
    o = torch.einsum("bhij,bjhd->bihd", a, v).reshape(B, S, H * D)
    return o @ p["out.weight"].T, h, x, residual, p


def rel(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().norm())


@pytest.mark.parametrize("window,ragged", [(0, False), (13, False), (0, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_against_plain(window, ragged, dtype):
    """With a generator for every token PAMM's weight gradient is exact, so all
    gradients have to be the plain ones: to sums of fp32 products (1e-5, over
    contractions of at most 192), or to bf16's 2^-8 through the six roundings
    between a loss and the input (2e-2)."""
    torch.manual_seed(1)
    tol = 1e-5 if dtype == torch.float32 else 2e-2
    B, S, dim = 2, 45, 96
    block = PammAttentionBlock(dim, 4, 2, head_dim=24, window=window, ratio=1, device="cuda", dtype=dtype)
    with torch.no_grad():
        block.norm.weight.copy_(1 + 0.1 * torch.randn(dim))
    x = torch.randn(B, S, dim, device="cuda").to(dtype).requires_grad_(True)
    r = torch.randn(B, S, dim, device="cuda").to(dtype).requires_grad_(True)
    lengths = torch.tensor([45, 20], dtype=torch.int32, device="cuda") if ragged else None
    out, h = block(x, r, lengths)
    g, gh = torch.randn(B, S, dim, device="cuda").to(dtype), torch.randn(B, S, dim, device="cuda").to(dtype)
    if ragged:
        g[1, 20:] = 0
    ((out * g).sum() + (h * gh).sum()).backward()
    want, hw, xw, rw, p = plain_block(block, x, r, lengths.cpu() if ragged else None)
    ((want * g.double().cpu()).sum() + (hw * gh.double().cpu()).sum()).backward()
    assert rel(out, want) < tol and rel(h, hw) < tol
    for name, got, ref in [("x", x.grad, xw.grad), ("residual", r.grad, rw.grad)] + [
            (n, t.grad, p[n].grad) for n, t in block.named_parameters()]:
        assert rel(got, ref) < tol, (name, rel(got, ref))


def test_wrappers_take_any_gradient_layout():
    torch.manual_seed(2)
    q, k, v = (torch.randn(2, 33, h, 32, device="cuda", requires_grad=True) for h in (4, 2, 2))
    o = differentiable_attention(q, k, v, causal=True, window=9)
    g = torch.randn(2, 32, 4, 33, device="cuda").permute(0, 3, 2, 1)  # neither contiguous nor rows of heads
    a = torch.autograd.grad(o, (q, k, v), g, retain_graph=True)
    b = torch.autograd.grad(o, (q, k, v), g.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    norm = AddRMSNorm(33, device="cuda")  # rows off 16 bytes
    x, r = torch.randn(3, 5, 33, device="cuda", requires_grad=True), torch.randn(3, 5, 33, device="cuda")
    y, h = norm(x, r)
    gy = torch.randn(33, 5, 3, device="cuda").permute(2, 1, 0)
    (dx,) = torch.autograd.grad(y, x, gy, retain_graph=True)
    (dx2,) = torch.autograd.grad(y, x, gy.contiguous(), retain_graph=True)
    assert torch.equal(dx, dx2)
    (dh,) = torch.autograd.grad(h.sum(), x)  # y not used at all
    assert torch.equal(dh, torch.ones_like(dh))
    y1, h1 = norm(x)
    assert h1 is x
    y1.sum().backward()
    assert x.grad is not None


@pytest.mark.parametrize("window", [0, 7])
def test_decoding_is_the_forward_pass(window):
    torch.manual_seed(3)
    B, S, dim = 3, 60, 128
    block = PammAttentionBlock(dim, 4, 2, window=window, device="cuda").eval()
    x, r = torch.randn(B, S, dim, device="cuda"), torch.randn(B, S, dim, device="cuda")
    with torch.no_grad():
        want, _ = block(x, r)
    cache = block.cache(B, S)
    got = [block.step(x[:, :17], r[:, :17], cache)[0], block.step(x[:, 17:40], r[:, 17:40], cache)[0]]
    got += [block.step(x[:, i:i + 1], r[:, i:i + 1], cache)[0] for i in range(40, S)]
    assert rel(torch.cat(got, 1), want) < 1e-5
    with pytest.raises(ValueError):
        block.step(x[:, :1], r[:, :1], cache)


def test_eight_bit_step():
    """8-bit operands are off by 2^-4 at most, at random: over the 128 terms of
    a product the error stays below 2^-4 of its size, and what follows does not
    enlarge it by more than a factor of 2."""
    torch.manual_seed(4)
    B, S, dim = 2, 48, 128
    block = PammAttentionBlock(dim, 4, 2, device="cuda", dtype=torch.bfloat16).eval()
    x, r = (torch.randn(B, S, dim, device="cuda").bfloat16() for _ in range(2))
    a, b = block.cache(B, S), block.cache(B, S)
    want, h = block.step(x, r, a)
    got, h8 = block.step(x, r, b, eight_bits=True)
    assert torch.equal(h, h8)
    assert rel(got, want) < 2.0 ** -3
    got, _ = block.step(x[:, :1], r[:, :1], KVCache(B, 4, 2, 32), eight_bits=True)
    assert torch.isfinite(got).all()


def test_clipping_is_torch_s():
    torch.manual_seed(5)
    a = [torch.nn.Parameter(torch.randn(s, device="cuda")) for s in ((40, 30), (7,), (3, 5, 11))]
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    for p, q in zip(a, b):
        p.grad = torch.randn_like(p)
        q.grad = p.grad.clone()
    n = pamm.clip_grad_norm([p.grad for p in a], 1.5)
    m = torch.nn.utils.clip_grad_norm_(b, 1.5)
    assert abs(float(n) - float(m)) < 1e-5 * float(m)
    assert all(torch.allclose(p.grad, q.grad, rtol=1e-5, atol=0) for p, q in zip(a, b))


def test_example_learns():
    res = run(steps=8, batch=2, seq=256, dim=256, heads=4, ratio=16, decode=8)
    assert res["losses"][-1] < res["losses"][0]
    assert all(math.isfinite(x) for x in res["gradient_norms"])
    assert res["decode_against_forward"] < 2e-2
