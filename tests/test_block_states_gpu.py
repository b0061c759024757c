"""GPU: the block's layers after something they depend on has changed."""
import pytest
import torch

from activation_compression_pamm_amd.block import PammAttentionBlock

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("change", ["optimizer", "data", "load_state_dict", "new parameter"])
def test_eight_bit_steps_follow_the_weight(change):
    """However the weight changes, the next step in 8 bits is that of the new
    weight, bit by bit what a block that has known no other gives."""
    torch.manual_seed(6)
    B, S, dim = 2, 32, 128
    block, other = (PammAttentionBlock(dim, 4, 2, device="cuda", dtype=torch.bfloat16).eval() for _ in range(2))
    x = torch.randn(B, S, dim, device="cuda").bfloat16()
    old, _ = block.step(x, None, block.cache(B, S), eight_bits=True)
    new = torch.randn_like(block.qkv.weight) / dim ** 0.5
    if change == "optimizer":
        opt = torch.optim.SGD([block.qkv.weight], lr=1.0)
        block.qkv.weight.grad = block.qkv.weight.detach() - new
        opt.step()
    elif change == "data":
        block.qkv.weight.data.copy_(new)
    elif change == "load_state_dict":
        block.load_state_dict(dict(block.state_dict(), **{"qkv.weight": new}))
    else:
        block.qkv.weight = torch.nn.Parameter(new)
    other.load_state_dict(block.state_dict())
    got, _ = block.step(x, None, block.cache(B, S), eight_bits=True)
    want, _ = other.step(x, None, other.cache(B, S), eight_bits=True)
    full, _ = block.step(x, None, block.cache(B, S))
    assert rel(old, full) > 0.5
    assert torch.equal(got, want) and rel(got, full) < 2.0 ** -3


def test_eight_bit_weights_kept_by_the_caller():
    """quantize_qkv() gives the weight as it is, for steps until it changes."""
    torch.manual_seed(7)
    block = PammAttentionBlock(128, 4, 2, device="cuda", dtype=torch.bfloat16).eval()
    x = torch.randn(2, 16, 128, device="cuda").bfloat16()
    kept = block.quantize_qkv()
    a, _ = block.step(x, None, block.cache(2, 16), eight_bits=kept)
    b, _ = block.step(x, None, block.cache(2, 16), eight_bits=True)
    assert torch.equal(a, b)
    block.qkv.weight.data.mul_(2)
    c, _ = block.step(x, None, block.cache(2, 16), eight_bits=kept)
    assert torch.equal(a, c)


def layers():
    from activation_compression_pamm_amd.block import AddRMSNorm, PackedAttentionFunction, differentiable_attention

    g = torch.Generator(device="cuda").manual_seed(8)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda", requires_grad=True)

    q, k, v, qkv, x = r(2, 20, 4, 32), r(2, 20, 2, 32), r(2, 20, 2, 32), r(2, 20, 8, 32), r(3, 5, 64)
    norm = AddRMSNorm(64, device="cuda")
    return {"attention": (q, differentiable_attention(q, k, v, causal=True)),
            "packed": (qkv, PackedAttentionFunction.apply(qkv, 4, 2, True, 0, None, None)),
            "norm": (x, norm(x)[0]), "residual": (x, norm(x, r(3, 5, 64))[0])}


@pytest.mark.parametrize("name", ["attention", "packed", "norm", "residual"])
def test_second_derivatives_are_refused(name):
    """The backward passes have no gradient of their own; one that takes part in
    a loss has to say so instead of counting as a constant."""
    x, y = layers()[name]
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    assert g.requires_grad
    with pytest.raises(RuntimeError, match="once_differentiable|differentiating twice"):
        (g.square().sum() + x.sum()).backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_at_any_address(dtype):
    """A contiguous gradient whose rows start off 16 bytes, as a view of a flat buffer."""
    from activation_compression_pamm_amd.block import AddRMSNorm, PackedAttentionFunction, differentiable_attention

    torch.manual_seed(9)

    def off(like):
        flat = torch.randn(1 + like.numel(), device="cuda").to(dtype)
        view = flat[1:].view(like.shape)
        assert view.is_contiguous() and view.data_ptr() % 16
        return view

    def r(*shape):
        return torch.randn(*shape, device="cuda").to(dtype).requires_grad_(True)

    q, k, v, qkv, x = r(2, 33, 4, 32), r(2, 33, 2, 32), r(2, 33, 2, 32), r(2, 33, 8, 32), r(3, 5, 64)
    norm = AddRMSNorm(64, device="cuda", dtype=dtype)
    for y, inputs in ((differentiable_attention(q, k, v, causal=True), (q, k, v)),
                      (PackedAttentionFunction.apply(qkv, 4, 2, True, 0, None, None), (qkv,)), (norm(x)[0], (x,))):
        g = off(y)
        a = torch.autograd.grad(y, inputs, g, retain_graph=True)
        b = torch.autograd.grad(y, inputs, g.clone())
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("packed", [False, True])
def test_lengths_changed_before_the_backward_pass(packed):
    """The backward pass needs the lengths of the forward pass: where they were
    written over meanwhile it is refused, like any saved tensor's."""
    from activation_compression_pamm_amd.block import PackedAttentionFunction, differentiable_attention

    torch.manual_seed(10)
    n = torch.tensor([33, 12], dtype=torch.int32, device="cuda")
    qkv = torch.randn(2, 33, 8, 32, device="cuda", requires_grad=True)

    def forward():
        if packed:
            return PackedAttentionFunction.apply(qkv, 4, 2, True, 0, None, n)
        return differentiable_attention(*qkv.split([4, 2, 2], dim=2), causal=True, q_len=n, kv_len=n)

    (want,) = torch.autograd.grad(forward().sum(), qkv)
    assert not want[1, 12:].any() and want[1, :12].any()
    y = forward()
    n.sub_(5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y.sum(), qkv)
