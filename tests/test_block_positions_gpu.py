"""GPU: the attention block with rotary positions, norms of queries and keys and
a cache in 8 bits, against a plain 64-bit one, and its operators in captured
graphs."""
import math

import pytest
import torch

import activation_compression_pamm_amd as pamm
from activation_compression_pamm_amd.block import KVCache8, PammAttentionBlock, run
from test_attention_gpu import lens, say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    return float((a - b).norm() / b.norm())


def plain_turn(x, pos, f, interleaved, magnitude):
    t = pos[:, :, None, None].double() * f
    c, s = magnitude * t.cos(), magnitude * t.sin()
    R = 2 * f.shape[0]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * c - b * s, a * s + b * c
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), x[..., R:]], -1)


def plain_block(block, x, residual, lengths, pos):
    """The block's definition on CPU in 64 bits, with gradients by autograd."""
    p = {n: t.detach().double().cpu().requires_grad_(True) for n, t in block.named_parameters()}
    x, residual = x.detach().double().cpu().requires_grad_(True), residual.detach().double().cpu().requires_grad_(True)
    h = x + residual
    norm = lambda t, w: t / torch.sqrt(t.square().mean(-1, keepdim=True) + block.norm.eps) * w
    B, S, _ = x.shape
    H, K, D = block.heads, block.heads_kv, block.head_dim
    q, k, v = (norm(h, p["norm.weight"]) @ p["qkv.weight"].T).view(B, S, H + 2 * K, D).split([H, K, K], dim=2)
    if block.q_norm is not None:
        q, k = norm(q, p["q_norm"]), norm(k, p["k_norm"])
    if block.rotary_dim:
        f = block._inv_freq.cpu()
        q, k = (plain_turn(t, pos, f, block.interleaved, block.magnitude) for t in (q, k))
    k, v = k.repeat_interleave(H // K, 2), v.repeat_interleave(H // K, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    i, j = torch.arange(S)[:, None], torch.arange(S)[None]
    m = (j <= i) & ((j > i - block.window) | (block.window == 0))
    m = m[None] & (i[None] < lengths[:, None, None]) & (j[None] < lengths[:, None, None])
    a = torch.softmax(s.masked_fill(~m[:, None], -1e300), -1) * m[:, None]
    o = torch.einsum("bhij,bjhd->bihd", a, v).reshape(B, S, H * D)
    return o @ p["out.weight"].T, h, x, residual, p


@pytest.mark.parametrize("qk_norm,rotary,kw", [
    (False, True, {}), (True, 0, {}), (True, True, {"rotary_interleaved": True}), (True, 12, {"window": 13}),
    (False, 16, {"rotary_interleaved": True, "rotary_base": 500.0,
                 "rotary_scaling": {"scaling": "yarn", "factor": 4.0, "original_length": 64}})])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ragged", [False, True])
def test_block_against_plain(qk_norm, rotary, kw, dtype, ragged):
    """With a generator for every token PAMM's weight gradient is exact, so all gradients have to be the plain ones:
    to sums of fp32 products (2e-5, over contractions of at most 192, the norms of queries and keys among them),
    or to bf16's 2^-8 through the seven roundings between a loss and the input (2.5e-2)."""
    say("block", qk_norm, rotary, kw, dtype, ragged)
    torch.manual_seed(1)
    tol = 2e-5 if dtype == torch.float32 else 2.5e-2
    B, S, dim = 2, 45, 96
    block = PammAttentionBlock(dim, 4, 2, head_dim=24, ratio=1, qk_norm=qk_norm, rotary=rotary, device="cuda", dtype=dtype,
                               **kw)
    with torch.no_grad():
        block.norm.weight.copy_(1 + 0.1 * torch.randn(dim))
        if qk_norm:
            block.q_norm.copy_(1.5 + 0.1 * torch.randn(24))
            block.k_norm.copy_(1 + 0.1 * torch.randn(24))
    x = torch.randn(B, S, dim, device="cuda").to(dtype).requires_grad_(True)
    r = torch.randn(B, S, dim, device="cuda").to(dtype).requires_grad_(True)
    lengths = lens([45, 20]) if ragged else None
    positions = torch.arange(S, device="cuda")[None] + torch.tensor([[3], [100000]], device="cuda") if ragged and rotary else None
    out, h = block(x, r, lengths, positions)
    g, gh = torch.randn(B, S, dim, device="cuda").to(dtype), torch.randn(B, S, dim, device="cuda").to(dtype)
    if ragged:
        g[1, 20:] = 0
    ((out * g).sum() + (h * gh).sum()).backward()
    pos = positions.cpu() if positions is not None else torch.arange(S)[None].expand(B, -1)
    want, hw, xw, rw, p = plain_block(block, x, r, lengths.cpu() if ragged else torch.tensor([S, S]), pos)
    ((want * g.double().cpu()).sum() + (hw * gh.double().cpu()).sum()).backward()
    assert rel(out, want) < tol and rel(h, hw) < tol
    for name, got, ref in [("x", x.grad, xw.grad), ("residual", r.grad, rw.grad)] + [
            (n, t.grad, p[n].grad) for n, t in block.named_parameters()]:
        assert rel(got, ref) < tol, (name, rel(got, ref))


@pytest.mark.parametrize("kw", [{"rotary": True}, {"qk_norm": True}, {"rotary": 16, "qk_norm": True, "window": 7}])
@pytest.mark.parametrize("cache8", [False, True])
def test_decoding_is_the_forward_pass(kw, cache8):
    """Positions follow the cache's lengths.  8-bit keys and values are off by 2^-4 at most, at random, which an
    average over them and a score's sum of 32 terms do not enlarge."""
    say("decode", kw, cache8)
    torch.manual_seed(3)
    B, S, dim = 3, 100, 128
    block = PammAttentionBlock(dim, 4, 2, device="cuda", **kw).eval()
    x, r = torch.randn(B, S, dim, device="cuda"), torch.randn(B, S, dim, device="cuda")
    with torch.no_grad():
        want, _ = block(x, r)
    cache = block.cache(B, S, eight_bits=cache8, block=32)
    got = [block.step(x[:, :17], r[:, :17], cache)[0], block.step(x[:, 17:70], r[:, 17:70], cache)[0]]
    got += [block.step(x[:, i:i + 1], r[:, i:i + 1], cache)[0] for i in range(70, S)]
    assert rel(torch.cat(got, 1), want) < (2.0 ** -4 if cache8 else 1e-5)
    assert cache.used == S and cache.lengths.tolist() == [S] * B
    with pytest.raises(ValueError, match="do not fit"):
        block.step(x[:, :1], r[:, :1], cache)


def test_a_cast_block_keeps_its_angles():
    block = PammAttentionBlock(64, 2, rotary=True).to("cuda").bfloat16()
    assert block._frequencies(torch.device("cuda", 0)).dtype == torch.float64
    x = torch.randn(1, 5, 64, device="cuda").bfloat16()
    a, _ = block.eval()(x)
    b, _ = block(x, positions=torch.arange(5, device="cuda") + 12345678)  # only differences of positions matter
    assert rel(a, b) < 2e-2


def test_refusals():
    for kw in ({"rotary": 66}, {"rotary": -2}, {"rotary": 7}):
        with pytest.raises(ValueError):
            PammAttentionBlock(64, 2, head_dim=64, **kw)
    block = PammAttentionBlock(64, 2, device="cuda")
    with pytest.raises(ValueError, match="positions"):
        block(torch.zeros(1, 3, 64, device="cuda"), positions=torch.arange(3, device="cuda"))
    cache = KVCache8(2, 64, 1, 16)
    for k, v in (((2, 65, 1, 16), None), ((1, 2, 1, 16), None), ((2, 2, 1, 16), (2, 1, 1, 16)), ((2, 2, 16), None)):
        x, y = (torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in (k, v or k))
        with pytest.raises(ValueError):
            cache.append(x, y)
    assert cache.used == 0 and not cache.lengths.any()
    with pytest.raises(TypeError):
        cache.append(torch.ones(2, 1, 1, 16, device="cuda"), torch.ones(2, 1, 1, 16, device="cuda"))


def test_positions_without_a_rotation_are_refused():
    block = PammAttentionBlock(64, 2, qk_norm=True, device="cuda")
    with pytest.raises(ValueError, match="positions"):
        block(torch.zeros(1, 3, 64, device="cuda"), positions=torch.arange(3, device="cuda"))


def test_second_derivatives_are_refused():
    block = PammAttentionBlock(64, 2, rotary=True, qk_norm=True, device="cuda")
    x = torch.randn(1, 4, 64, device="cuda", requires_grad=True)
    out, _ = block(x)
    (g,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def operators():
    """name -> (inputs, call on them)"""
    g = torch.Generator(device="cuda").manual_seed(17)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    f = pamm.rotary_frequencies(64)[0]
    off = lens([900, 17])

    def norm(q, k, w, dq, dk):
        return (*pamm.qk_norm_rotary(q, k, w, w, f, offset=off), pamm.rotary(q, f, offset=off),
                *pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, offset=off))

    c = pamm.CacheFP8.empty(2, 1024, 2, 64)
    start = lens([900, 63])
    pamm.cache_append_fp8(c, r(2, 900, 2, 64), r(2, 900, 2, 64), lens([0, 0]), new_len=start)

    def token(q, k, v):
        n = start.clone()
        pamm.cache_append_fp8(c, k, v, n)
        o, lse = pamm.attention_fp8(q, c, n, causal=True)
        return o, lse, n.float()

    def chunk(q):
        return pamm.attention_fp8(q, c, start, causal=True, window=300)

    return {"norm": ((r(2, 300, 4, 64), r(2, 300, 2, 64), r(64), r(2, 300, 4, 64), r(2, 300, 2, 64)), norm),
            "token": ((r(2, 1, 8, 64), r(2, 1, 2, 64), r(2, 1, 2, 64)), token),
            "chunk": ((r(2, 60, 8, 64),), chunk)}


@pytest.mark.parametrize("name", ["norm", "token", "chunk"])
def test_replays_are_the_eager_results(name):
    say("graph", name)
    inputs, call = operators()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*inputs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*inputs)
    for i in range(4):
        for t in inputs:
            t.mul_(1.25 if i % 2 else -0.75)
        want = call(*inputs)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_a_captured_step_decodes():
    """One captured step of the block, replayed: lengths move on the GPU, so each replay is the next token."""
    torch.manual_seed(5)
    block = PammAttentionBlock(128, 4, 2, rotary=True, qk_norm=True, device="cuda", dtype=torch.bfloat16).eval()
    x = torch.randn(2, 50, 128, device="cuda").bfloat16()
    eager, cache = block.cache(2, 64, eight_bits=True, block=32), block.cache(2, 64, eight_bits=True, block=32)
    block.step(x[:, :20], None, eager)
    block.step(x[:, :20], None, cache)
    want = [block.step(x[:, i:i + 1], None, eager)[0].clone() for i in range(20, 50)]
    token = x[:, 20:21].clone()
    cache.used = 64  # the captured call attends over the whole room, up to the lengths
    side, warm = torch.cuda.Stream(), block.cache(2, 64, eight_bits=True, block=32)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(token, None, warm)
    torch.cuda.current_stream().wait_stream(side)
    cache.used = 63
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(token, None, cache)
    for i in range(20, 50):
        token.copy_(x[:, i:i + 1])
        graph.replay()
        torch.cuda.synchronize()
        # the same kernels on the same keys
        assert rel(out, want[i - 20]) < 1e-2, i
    assert cache.lengths.tolist() == [50, 50]


def test_example_runs():
    res = run(steps=2, batch=2, seq=256, dim=256, heads=4, ratio=16, decode=8, rotary=True, qk_norm=True, cache8=True)
    assert all(math.isfinite(x) for x in res["losses"] + res["gradient_norms"])
    assert res["decode_against_forward"] < 2.0 ** -3
