"""GPU: the 8-bit output of the norm is the nearest to its definition, ties included."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import dev, host, say, values
from test_norm_clip_gpu import rows

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("n,d", [(7, 2550), (16, 1300), (300, 768), (1100, 1000), (3, 4096), (5, 8)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-12, 1e12])
def test_bf16_rows_are_rounded_exactly(n, d, residual, size):
    """y / scale = 448 h w / max|h w|: 1/rms cancels, and with bf16 h and w both
    products have 16 bits.  A quotient of 7 x 16-bit and 16-bit integers that is no
    tie of the 8-bit type (5 bits) is 2^-21 of it away from one at least, and one
    that is a tie has an exact fp32 value, so fp32 suffices to round every element
    as the definition does, to even where it is a tie."""
    say("8-bit rows", n, d, residual, size)
    rng = np.random.default_rng(n + d)
    x = bo.to_bf16(values(rng, (n, d), "bf16") * size)
    x[:, ::max(1, d // 5)] *= 8
    r = bo.to_bf16(values(rng, (n, d), "bf16", 2.0) * size) if residual else None
    w = bo.to_bf16(1 + 0.2 * rng.standard_normal(d))
    q, scale, h, rstd = pamm.add_rms_norm_fp8(rows(x, "bf16"), dev(w, "bf16"), rows(r, "bf16") if residual else None)
    p = host(h) * w
    want = bo.e4m3(448 * p / np.abs(p).max(1, keepdims=True))
    assert np.array_equal(host(q.float()), want)
    top = np.abs(p * host(rstd)[:, None]).max(1) / 448
    assert (np.abs(host(scale) - top) <= 4 * bo.U * top).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extremes(dtype):
    """Weights and rows at the ends of the range, rows of zeros, what is not finite."""
    say("8-bit extremes", dtype)
    d = 64
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.ones(8, d, device="cuda")
    x[1] *= 1e18
    x[2] *= 1e-18
    x[3] = 0
    x[4, 7] = float("nan")
    x[5, 7] = float("-inf")
    x[6, ::2] = 0
    w = torch.ones(d, device="cuda")
    for factor in (1.0, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126, 2.0 ** 126):
        q, scale, _, rstd = pamm.add_rms_norm_fp8(x.to(t), (w * factor).to(t))
        y, _, _ = pamm.add_rms_norm(x.to(t), (w * factor).to(t))
        q = q.float()
        assert torch.isnan(q[4]).all() and torch.isnan(q[5, 7]) and not q[5][torch.arange(d, device="cuda") != 7].any()
        assert not q[3].any() and float(scale[3]) == 2.0 ** -126
        for i in (0, 1, 2, 6, 7):
            back, want = q[i].double() * scale[i].double(), y[i].double()
            top = y[i].double().abs().max()
            # what is not 0 in a row has one size, so q is 0 or 448 but for the roundings of y and the
            # scale; a row with the smallest scale has smaller values, rounded to half a step, 2^-4 of
            # them or 2^-10 scales
            r = 2.0 ** -4 if float(scale[i]) == 2.0 ** -126 else 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
            assert (back - want).abs().max() <= r * top + 2.0 ** -136, (factor, i)
            assert abs(float(scale[i]) - max(float(top) / 448, 2.0 ** -126)) <= 2.0 ** -8 * float(scale[i])
    w[9] = float("inf")
    q, scale, _, _ = pamm.add_rms_norm_fp8(x[:1].to(t), w.to(t))
    q = q.float()
    assert torch.isnan(q[0, 9]) and not q[0][torch.arange(d, device="cuda") != 9].any() and torch.isinf(scale).all()
