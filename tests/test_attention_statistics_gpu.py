"""GPU: attention's running softmax statistics where they move, and the
precision of its gradients, against the 64-bit definition (tests/block_oracle.py)."""
import math

import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import close, dev, lens, say, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def compare(q, k, v, do, dtype, **kw):
    ref = bo.attention(q, k, v, do, dtype=dtype, **kw)
    gk = dict(kw, q_len=lens(kw.get("q_len")), kv_len=lens(kw.get("kv_len")))
    qd, kd, vd, dod = (dev(x, dtype) for x in (q, k, v, do))
    o, lse = pamm.attention(qd, kd, vd, **gk)
    close("o", o, ref["o"], ref["o_tol"])
    close("lse", lse, ref["lse"], ref["lse_tol"])
    for n, t in zip(("dq", "dk", "dv"), pamm.attention_backward(dod, qd, kd, vd, o, lse, **gk)):
        close(n, t, ref[n], ref[n + "_tol"])


# Factors of the keys along their sequence: the largest score of a block of 32
# rises or falls by far more than 2^8 from block to block, stays, or leaps once.
PATHS = {"rising": lambda n: np.linspace(0.1, 20.0, n), "falling": lambda n: np.linspace(20.0, 0.1, n),
         "leap": lambda n: np.where(np.arange(n) == n // 2, 40.0, 1.0),
         "late": lambda n: np.where(np.arange(n) == n - 1, 40.0, 0.01)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("Sq,Sk,D,kw", [(70, 200, 64, {}), (150, 150, 64, {"causal": True}), (200, 200, 32, {"causal": True, "window": 37}),
                                        (70, 200, 128, {"causal": True}), (1, 700, 64, {}), (40, 1500, 64, {})])
def test_scores_that_rise_and_fall(dtype, path, Sq, Sk, D, kw):
    say("path", dtype, path, Sq, Sk, D, kw)
    rng = np.random.default_rng(3)
    q, do = values(rng, (2, Sq, 2, D), dtype), values(rng, (2, Sq, 2, D), dtype)
    k, v = values(rng, (2, Sk, 1, D), dtype), values(rng, (2, Sk, 1, D), dtype)
    k = k * PATHS[path](Sk)[None, :, None, None]
    compare(q, bo.to_bf16(k) if dtype == "bf16" else k.astype(np.float32).astype(np.float64), v, do, dtype, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_from_zero(dtype, sign, D):
    """Every score near -1000 or 1000 of one sequence, near 0 of the other."""
    say("far", dtype, sign, D)
    rng = np.random.default_rng(4)
    q, do = values(rng, (2, 90, 2, D), dtype), values(rng, (2, 90, 2, D), dtype)
    k, v = values(rng, (2, 90, 2, D), dtype), values(rng, (2, 90, 2, D), dtype)
    q[0, ..., 0], k[0, ..., 0] = 64.0, sign * 16.0 * math.sqrt(D)
    k = bo.to_bf16(k) if dtype == "bf16" else k.astype(np.float32).astype(np.float64)
    compare(q, k, v, do, dtype, causal=True)


@pytest.mark.parametrize("S,H,Hkv,D,window", [(20, 8, 8, 64, 0), (300, 8, 8, 64, 0), (300, 8, 2, 128, 0), (300, 4, 4, 96, 0),
                                              (500, 8, 8, 64, 8), (500, 8, 2, 128, 16), (33, 4, 4, 32, 12)])
def test_precision_of_bf16_gradients(S, H, Hkv, D, window):
    """Beside the rounding of the result, whose relative error an exact gradient
    has too, dS (for dv: P) is rounded once, independently and as finely: sqrt(2)
    times the exact gradient's error.  1.5 leaves the rest a quarter of one such
    error's square, which the rounding of o in delta exceeds where rows see few
    keys, if it is not corrected."""
    say("precision", S, H, Hkv, D, window)
    rng = np.random.default_rng(5)
    q, do = values(rng, (2, S, H, D), "bf16"), values(rng, (2, S, H, D), "bf16")
    k, v = values(rng, (2, S, Hkv, D), "bf16"), values(rng, (2, S, Hkv, D), "bf16")
    ref = bo.attention(q, k, v, do, dtype="bf16", causal=True, window=window)
    qd, kd, vd, dod = (dev(x, "bf16") for x in (q, k, v, do))
    o, lse = pamm.attention(qd, kd, vd, causal=True, window=window)
    for n, t in zip(("dq", "dk", "dv"), pamm.attention_backward(dod, qd, kd, vd, o, lse, causal=True, window=window)):
        want = ref[n]
        off = np.linalg.norm(t.double().cpu().numpy() - want)
        exact = np.linalg.norm(bo.to_bf16(want) - want)
        assert off <= 1.5 * exact, f"{n}: {off / exact:.3f} times the exact gradient's rounding"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Sq", [1, 40])
@pytest.mark.parametrize("stride", [0, 64, 1 << 35])
def test_stride_of_a_single_key(dtype, Sq, stride):
    """A sequence of one key has no distance to the next: no tile's further rows
    are that key again, whose infinity would meet their probability 0."""
    say("single key", dtype, Sq, stride)
    rng = np.random.default_rng(6)
    q = dev(values(rng, (1, Sq, 2, 64), dtype), dtype)
    flat = dev(values(rng, (2, 128), dtype), dtype)
    flat[1, 5] = math.inf
    k, v = (torch.as_strided(t, (1, 1, 2, 64), (stride, stride, 64, 1)) for t in flat)
    o, lse = pamm.attention(q, k, v)
    same, fin = v.expand(1, Sq, 2, 64).double(), torch.isfinite(v).expand(1, Sq, 2, 64)
    assert torch.equal(torch.isfinite(o), fin) and torch.equal(o.double()[~fin], same[~fin])
    assert ((o.double() - same)[fin].abs() <= same[fin].abs() * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -21)).all()
    want = (q.double() * k.double()).sum(-1).transpose(1, 2) / 8.0
    assert (lse.double() - want).abs().max() < 1e-4


@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 64), (16, 8, 128), (8, 8, 96), (16, 16, 32)])
def test_every_lane_has_the_corrected_delta(H, Hkv, D):
    """In one launch, delta's correction is formed by the lanes of the first 16
    keys of a block and used by all.  Here the two keys behind those have all of
    the weight, so that the rounding of o in delta shows: uncorrected it adds half
    of an exact gradient's squared error or more to its own and that of dS (1.58
    times its error), corrected the bound of test_precision_of_bf16_gradients holds."""
    say("corrected delta", H, Hkv, D)
    rng = np.random.default_rng(11)
    B, Sq, Sk = 16, 40, 18
    q, do = values(rng, (B, Sq, H, D), "bf16"), values(rng, (B, Sq, H, D), "bf16")
    k, v = values(rng, (B, Sk, Hkv, D), "bf16"), values(rng, (B, Sk, Hkv, D), "bf16")
    q[..., 0], k[:, :, :, 0] = 2.0, 0.0
    k[:, :16, :, 0] = -32.0 * math.sqrt(D) // 1  # scores near -64
    k = bo.to_bf16(k)
    ref = bo.attention(q, k, v, do, dtype="bf16")
    qd, kd, vd, dod = (dev(x, "bf16") for x in (q, k, v, do))
    o, lse = pamm.attention(qd, kd, vd)
    got = pamm.attention_backward(dod, qd, kd, vd, o, lse)[1].double().cpu().numpy()[:, 16:]
    want = ref["dk"][:, 16:]
    off, exact = np.linalg.norm(got - want), np.linalg.norm(bo.to_bf16(want) - want)
    assert off <= 1.5 * exact, f"{off / exact:.3f} times the exact gradient's rounding"


@pytest.mark.parametrize("B,S,H,Hkv,D,kw", [(4, 215, 2, 2, 96, {}), (1, 31, 8, 4, 128, {"causal": True}), (2, 600, 2, 2, 64, {}),
                                            (2, 333, 4, 2, 40, {"causal": True}), (1, 512, 2, 1, 128, {"scale": -0.02})])
def test_precision_of_fp32_gradients(B, S, H, Hkv, D, kw):
    """P = 2^x with x = log2(e) (s - lse): x, lse and its multiple are rounded at
    their own size, |x| <= 16 and |lse| log2(e) <= 16 here, each to 2^-21 at most and
    evenly: three of 2^-21 ln(2) / sqrt(3) add up, squared, to 3.3e-7; the scores'
    products, |s| <= 8, and those of dout add less, and sums over keys at most as
    much again: 1e-6 of the gradient.  Scores summed on top of lse / scale instead
    are rounded at its size in each of their D / 2 steps."""
    say("fp32 gradients", B, S, H, Hkv, D, kw)
    rng = np.random.default_rng(16)
    q, do = values(rng, (B, S, H, D), "f32"), values(rng, (B, S, H, D), "f32")
    k, v = values(rng, (B, S, Hkv, D), "f32"), values(rng, (B, S, Hkv, D), "f32")
    ref = bo.attention(q, k, v, do, **kw)
    qd, kd, vd, dod = (dev(x, "f32") for x in (q, k, v, do))
    o, lse = pamm.attention(qd, kd, vd, **kw)
    for n, t in zip(("dq", "dk", "dv"), pamm.attention_backward(dod, qd, kd, vd, o, lse, **kw)):
        off = np.linalg.norm(t.double().cpu().numpy() - ref[n]) / np.linalg.norm(ref[n])
        say(n, off)
        assert off <= 1e-6, f"{n}: {off:.3g}"


@pytest.mark.parametrize("S", [33, 35, 48, 64, 65, 70, 96])
@pytest.mark.parametrize("H,Hkv,D", [(16, 4, 32), (8, 2, 96), (4, 1, 128), (8, 8, 64)])
def test_precision_of_bf16_gradients_of_few_keys(S, H, Hkv, D):
    """The bound of test_precision_of_bf16_gradients where every query sees the
    same few keys, more than one tile of them."""
    say("few keys", S, H, Hkv, D)
    rng = np.random.default_rng(S)
    q, do = values(rng, (4, S, H, D), "bf16"), values(rng, (4, S, H, D), "bf16")
    k, v = values(rng, (4, S, Hkv, D), "bf16"), values(rng, (4, S, Hkv, D), "bf16")
    ref = bo.attention(q, k, v, do, dtype="bf16")
    qd, kd, vd, dod = (dev(x, "bf16") for x in (q, k, v, do))
    o, lse = pamm.attention(qd, kd, vd)
    for n, t in zip(("dq", "dk", "dv"), pamm.attention_backward(dod, qd, kd, vd, o, lse)):
        want = ref[n]
        off, exact = np.linalg.norm(t.double().cpu().numpy() - want), np.linalg.norm(bo.to_bf16(want) - want)
        assert off <= 1.5 * exact, f"{n}: {off / exact:.3f} times the exact gradient's rounding"
