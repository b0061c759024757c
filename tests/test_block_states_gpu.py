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
