"""GPU: clip_grad_norm at the ends of its limit's range."""
import math

import pytest
import torch

import activation_compression_pamm_amd as pamm

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def grads():
    g = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(700, 33, generator=g, device="cuda"), torch.randn(5001, generator=g, device="cuda").bfloat16()]


@pytest.mark.parametrize("limit", [math.inf, 1e39, 3.4028234663852886e38, 3e38])
def test_out_is_written_without_a_limit_in_reach(limit):
    """min(1, limit / (norm + eps)) is 1: out is the gradients, also as fp32."""
    g = grads()
    keep = [t.clone() for t in g]
    for dtypes in ([t.dtype for t in g], [torch.float32] * 2):
        out = [torch.full(t.shape, float("nan"), dtype=d, device="cuda") for t, d in zip(g, dtypes)]
        norm = pamm.clip_grad_norm(g, limit, out=out)
        assert torch.equal(norm, pamm.clip_grad_norm(g))
        for a, o in zip(g, out):
            assert torch.equal(o, a.to(o.dtype))
    assert torch.equal(pamm.clip_grad_norm(g, limit), norm)
    assert all(torch.equal(a, b) for a, b in zip(g, keep))


@pytest.mark.parametrize("limit", [1e39, 1.0])
def test_an_infinite_norm_under_any_finite_limit(limit):
    x = torch.tensor([1.0, float("inf"), -2.0], device="cuda")
    out = torch.empty_like(x)
    assert math.isinf(float(pamm.clip_grad_norm([x], limit, out=[out])))
    assert out[0] == 0 and torch.isnan(out[1]) and out[2] == 0
    assert math.isinf(float(pamm.clip_grad_norm([x], limit)))
    assert x[0] == 0 and torch.isnan(x[1]) and x[2] == 0


def test_limits_that_are_none():
    g = grads()
    for bad in (-math.inf, -1e39, math.nan):
        with pytest.raises(pamm.PammError):
            pamm.clip_grad_norm(g, bad)
        with pytest.raises(pamm.PammError):
            pamm.clip_grad_norm(g, bad, out=[torch.empty_like(t) for t in g])


def test_zero_gradients_under_a_limit_of_zero():
    """coef is 0 / 0 without eps; what is scaled is 0 all the same."""
    for eps in (0.0, 1e-6):
        x, out = torch.zeros(1000, device="cuda"), torch.full((1000,), 7.0, device="cuda")
        assert float(pamm.clip_grad_norm([x], 0.0, eps=eps, out=[out])) == 0.0
        assert float(pamm.clip_grad_norm([x], 0.0, eps=eps)) == 0.0
        assert not x.any() and not out.any()
        y = torch.full((1000,), 1e-30, device="cuda")
        pamm.clip_grad_norm([y], 0.0, eps=eps)
        assert not y.any()
