"""GPU: the residual addition with its RMS norm (forward, 8-bit output,
backward) and the global gradient norm with clipping, against plain 64-bit
definitions (bounds derived in tests/block_oracle.py)."""
import math
import sys

import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import DT, close, dev, host, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def rows(x, dtype):
    """On the device with rows a multiple of 16 bytes apart."""
    n, d = x.shape
    per = 8 if dtype == "bf16" else 4
    buf = torch.full((n, (d + per - 1) // per * per), float("nan"), dtype=DT[dtype], device="cuda")
    buf[:, :d] = dev(x, dtype)
    return buf[:, :d]


SIZES = [(1, 1), (3, 7), (5, 8), (4, 768), (7, 1000), (33, 65), (2, 4096), (1030, 512), (1100, 2048), (1025, 4097),
         (1, 16384), (3, 16381), (1030, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", SIZES + [(2, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dtype, n, d, residual):
    if dtype == "f32" and d > 16384:
        pytest.skip("longer than a row may be")
    rng = np.random.default_rng(n + d)
    say("norm", n, d, dtype, residual)
    x, dy, dh = (values(rng, (n, d), dtype, s) for s in (1.0, 1.0, 0.5))
    r = values(rng, (n, d), dtype, 2.0) if residual else None
    w = values(rng, (d,), dtype)
    ref = bo.add_rms_norm(x, w, r, dtype=dtype, dy=dy, dh=dh)
    xd, rd, wd = rows(x, dtype), rows(r, dtype) if residual else None, dev(w, dtype)
    y, h, rstd = pamm.add_rms_norm(xd, wd, rd)
    assert np.array_equal(host(h), ref["h"])
    close("rstd", rstd, ref["rstd"], ref["rstd_tol"])
    close("y", y, ref["y"], ref["y_tol"])
    q, scale, h8, rstd8 = pamm.add_rms_norm_fp8(xd, wd, rd)
    assert torch.equal(h8, h) and torch.equal(rstd8, rstd)
    close("scale", scale, ref["scale"], ref["scale_tol"])
    # the 8-bit values are the nearest to y / scale: within half a step (2^-4
    # of the value, 2^-10 below 2^-6) and the error of the quotient
    want = ref["y"] / host(scale)[:, None]
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -6))) - 4)
    close("q", q.float(), want, step * (1 + 1e-4) + np.abs(want) * ref["scale_tol"][:, None] / ref["scale"][:, None] * 4)
    exact = bo.e4m3(want)
    assert (host(q.float()) != exact).mean() <= 0.01, "8-bit values differ from the nearest too often"
    dx, dw = pamm.add_rms_norm_backward(rows(dy, dtype), h, wd, rstd, dh=rows(dh, dtype))
    close("dx", dx, ref["dx"], ref["dx_tol"])
    close("dw", dw, ref["dw"], ref["dw_tol"])
    dx2, dw2 = pamm.add_rms_norm_backward(rows(dy, dtype), h, wd, rstd, dh=rows(dh, dtype))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    plain = bo.add_rms_norm(x, w, r, dtype=dtype, dy=dy)
    dx, _ = pamm.add_rms_norm_backward(rows(dy, dtype), h, wd, rstd)
    close("dx without dh", dx, plain["dx"], plain["dx_tol"])


def test_norm_in_place():
    rng = np.random.default_rng(0)
    x, r, w, dy = values(rng, (40, 256), "bf16"), values(rng, (40, 256), "bf16"), values(rng, (256,), "bf16"), values(
        rng, (40, 256), "bf16")
    y0, h0, rstd0 = pamm.add_rms_norm(dev(x, "bf16"), dev(w, "bf16"), dev(r, "bf16"))
    rd = dev(r, "bf16")
    y, h, rstd = pamm.add_rms_norm(dev(x, "bf16"), dev(w, "bf16"), rd, h=rd)
    assert h is rd and torch.equal(h, h0) and torch.equal(y, y0)
    want, _ = pamm.add_rms_norm_backward(dev(dy, "bf16"), h, dev(w, "bf16"), rstd, dh=dev(x, "bf16"))
    for which in ("dy", "dh"):
        a, b = dev(dy, "bf16"), dev(x, "bf16")
        got, _ = pamm.add_rms_norm_backward(a, h, dev(w, "bf16"), rstd, dh=b, dx=a if which == "dy" else b)
        assert torch.equal(got, want), which


def test_norm_rows_do_not_touch_each_other():
    x = torch.ones(6, 64, device="cuda")
    x[1, 3], x[2, 5], x[4] = float("nan"), float("inf"), 0.0
    w = torch.ones(64, device="cuda")
    y, _, rstd = pamm.add_rms_norm(x, w)
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 5]) and not y[2, :5].any()
    assert torch.allclose(y[[0, 3, 5]], torch.ones(3, 64, device="cuda"))
    assert not y[4].any()
    q, scale, _, _ = pamm.add_rms_norm_fp8(x, w)
    assert torch.isnan(q[1].float()).all() and torch.isnan(q[2, 5].float())
    assert not q[4].float().any() and float(scale[4]) == 2.0 ** -126
    assert bool((q[0].float() == 448).all())


def test_norm_gradient_against_differences():
    """Directional differences of the 64-bit definition; h = 1e-5 and third
    derivatives of order one leave ~1e-10 of the derivative."""
    rng = np.random.default_rng(1)
    n, d, h = 9, 100, 1e-5
    x, w, dy = values(rng, (n, d), "f32"), values(rng, (d,), "f32"), values(rng, (n, d), "f32")
    xd, wd = dev(x, "f32"), dev(w, "f32")
    _, hd, rstd = pamm.add_rms_norm(xd, wd)
    dx, dw = pamm.add_rms_norm_backward(dev(dy, "f32"), hd, wd, rstd)
    ref = bo.add_rms_norm(x, w, dy=dy)
    for got, tol, size, f in ((dx, ref["dx_tol"], (n, d), lambda t: bo.add_rms_norm(x + t, w)["y"]),
                              (dw, ref["dw_tol"], (d,), lambda t: bo.add_rms_norm(x, w + t)["y"])):
        way = rng.standard_normal(size)
        diff = ((f(h * way) * dy).sum() - (f(-h * way) * dy).sum()) / (2 * h)
        assert abs((host(got) * way).sum() - diff) <= (tol * np.abs(way)).sum() + 1e-6 * abs(diff)


def test_norm_refusals_and_empty():
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        pamm.add_rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        pamm.add_rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        pamm.add_rms_norm(x, w, torch.ones(4, 63, device="cuda"))
    with pytest.raises(ValueError):
        pamm.add_rms_norm(x.t(), w)
    with pytest.raises(ValueError):
        pamm.add_rms_norm(x, w, h=x)
    with pytest.raises(TypeError):
        pamm.add_rms_norm(x.half(), w.half())
    with pytest.raises(pamm.PammError):
        pamm.add_rms_norm(torch.ones(4, 70, device="cuda")[:, :64], w)  # rows off 16 bytes
    with pytest.raises(pamm.PammError):
        pamm.add_rms_norm(x, w, eps=-1.0)
    with pytest.raises(pamm.PammError):
        pamm.add_rms_norm(torch.ones(2, 16400, device="cuda"), torch.ones(16400, device="cuda"))
    y, h, rstd = pamm.add_rms_norm(x[:0], w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = pamm.add_rms_norm_backward(x[:0], x[:0], w, rstd)
    assert dx.shape == (0, 64) and not dw.any()


# -------------------------------------------------------------------- clipping

def grads_of(rng, shapes, dtypes, scale=1e-3):
    return [dev(values(rng, s, t, scale), t) for s, t in zip(shapes, dtypes)]


def ref_norm(grads):
    return math.sqrt(sum(float((host(g) ** 2).sum()) for g in grads))


def check_clip(grads, max_norm, outs=None):
    before = [host(g) for g in grads]
    norm = math.sqrt(sum(float((b ** 2).sum()) for b in before))
    got = pamm.clip_grad_norm(grads, max_norm, out=outs)
    assert abs(float(got) - norm) <= 2 * bo.U * norm  # summed in 64 bits, rounded once
    coef = min(1.0, max_norm / (norm + 1e-6))
    for b, o in zip(before, outs or grads):
        r = 2.0 ** -8 if o.dtype == torch.bfloat16 else bo.U
        close("clipped", o, coef * b, (r + 8 * bo.U) * np.abs(coef * b) + (2.0 ** -134 if r > bo.U else 2.0 ** -149))


@pytest.mark.parametrize("kind", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("over", [True, False])
def test_clip(kind, over):
    rng = np.random.default_rng(2)
    shapes = [(1,), (7,), (300, 5), (129, 257), (16384,), (16385,), (3, 50001), (0,), (64, 64, 3)]
    dtypes = [kind if kind != "mixed" else ("bf16", "f32")[i % 2] for i in range(len(shapes))]
    grads = grads_of(rng, shapes, dtypes)
    limit = ref_norm(grads) * (0.25 if over else 4.0)
    outs = [torch.full_like(g, float("nan")) for g in grads]
    check_clip(grads, limit, outs)
    wide = [torch.full(g.shape, float("nan"), device="cuda") for g in grads]
    check_clip(grads, limit, wide)
    narrow = [torch.full(g.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for g in grads]
    check_clip(grads, limit, narrow)
    kept = [g.clone() for g in grads]
    check_clip(grads, limit)
    assert over or all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_clip_many_tensors_and_odd_offsets():
    rng = np.random.default_rng(3)
    # pieces of a flat buffer at every alignment, with gaps, over several launches
    flat = dev(values(rng, (60000,), "bf16", 1e-2), "bf16")
    keep = flat.clone()
    grads, at = [], 0
    for i in range(150):
        n = 1 + (i * 37) % 300
        grads.append(flat[at:at + n])
        at += n + (i % 3)
    check_clip(grads, ref_norm(grads) * 0.5)
    covered = torch.zeros(60000, dtype=torch.bool, device="cuda")
    at = 0
    for i in range(150):
        n = 1 + (i * 37) % 300
        covered[at:at + n] = True
        at += n + (i % 3)
    assert torch.equal(flat[~covered], keep[~covered]), "a gap was written"


def test_clip_layouts():
    rng = np.random.default_rng(4)
    a = torch.empty(30, 20, device="cuda")[:, :17]  # padded rows
    a.copy_(dev(values(rng, (30, 17), "f32"), "f32"))
    b = dev(values(rng, (8, 9, 10), "f32"), "f32").permute(2, 0, 1)  # dense, another order
    wide = dev(values(rng, (25, 40), "bf16"), "bf16")
    c, d = wide[:, :11], wide[:, 11:]  # interleaved columns of one matrix
    grads = [a, None, b, c, d]
    given = [g for g in grads if g is not None]
    before = [host(g) for g in given]
    norm = pamm.clip_grad_norm(grads, 1.0)
    want = math.sqrt(sum(float((x ** 2).sum()) for x in before))
    assert abs(float(norm) - want) <= 2 * bo.U * want
    for x, g in zip(before, given):
        close("clipped", g, x / (want + 1e-6), (2.0 ** -8 + 8 * bo.U) * np.abs(x / want))
    out = [torch.empty(30, 17, device="cuda"), None, torch.empty_like(b), torch.empty_like(c), torch.empty_like(d)]
    check_clip(given, 0.5, [o for o in out if o is not None])


def test_clip_extremes():
    big = torch.full((1000,), 3e38, dtype=torch.bfloat16, device="cuda")
    small = torch.full((1000,), 1e-30, device="cuda")
    n = float(pamm.clip_grad_norm([small]))
    assert abs(n - 1e-30 * math.sqrt(1000)) <= 1e-6 * n  # its squares vanish in fp32
    assert math.isinf(float(pamm.clip_grad_norm([big])))  # the norm itself passes fp32
    half = torch.full((4,), 1e30, device="cuda")
    pamm.clip_grad_norm([half], 2.0)
    assert torch.allclose(half, torch.ones(4, device="cuda"))
    x = torch.tensor([1.0, float("inf"), -2.0], device="cuda")
    assert math.isinf(float(pamm.clip_grad_norm([x], 1.0)))
    assert x[0] == 0 and torch.isnan(x[1]) and x[2] == 0
    x = torch.tensor([1.0, float("nan")], device="cuda")
    assert math.isnan(float(pamm.clip_grad_norm([x], 1.0))) and torch.isnan(x).all()
    x = torch.zeros(5, device="cuda")
    assert float(pamm.clip_grad_norm([x], 1.0)) == 0.0 and not x.any()
    x = torch.ones(5, device="cuda")
    pamm.clip_grad_norm([x], 0.0)
    assert not x.any()


def test_clip_refusals():
    x = torch.ones(10, device="cuda")
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x, x], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x, x[5:]], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x[:6], x[1:2], x[4:8]], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x.expand(3, 10)], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x.cpu()], 1.0)
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x], 1.0, out=[torch.ones(9, device="cuda")])
    with pytest.raises(ValueError):
        pamm.clip_grad_norm([x], 1.0, out=[])
    with pytest.raises(TypeError):
        pamm.clip_grad_norm([x.double()], 1.0)
    with pytest.raises(pamm.PammError):
        pamm.clip_grad_norm([x], -1.0)
    with pytest.raises(pamm.PammError):
        pamm.clip_grad_norm([x], float("nan"))
    assert torch.equal(x, torch.ones(10, device="cuda"))
    assert float(pamm.clip_grad_norm([x, x])) == pytest.approx(math.sqrt(20))  # the norm alone writes nothing
