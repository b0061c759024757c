"""GPU: attention and its backward pass against the plain 64-bit definition
(tests/block_oracle.py, which also derives the bounds), at the sizes and masks
where they can go wrong, and against differences."""
import sys

import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def values(rng, shape, dtype, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32).astype(np.float64)
    return bo.to_bf16(x) if dtype == "bf16" else x


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", DT[dtype])


def host(t):
    return t.double().cpu().numpy()


def close(name, got, want, tol):
    got = host(got) if isinstance(got, torch.Tensor) else got
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), f"{name}: not finite in other places"
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    bad = ~(off <= tol + 1e-37) & fin
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside the bound, worst off "
                           f"{np.nanmax(np.where(bad, off, 0)):.3e} at {np.argwhere(bad)[0]}")


def lens(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def check(B, Sq, Sk, H, Hkv, D, dtype, *, backward=True, seed=0, arrange=None, **kw):
    rng = np.random.default_rng(seed)
    q, do = values(rng, (B, Sq, H, D), dtype), values(rng, (B, Sq, H, D), dtype)
    k, v = values(rng, (B, Sk, Hkv, D), dtype), values(rng, (B, Sk, Hkv, D), dtype)
    say("attention", B, Sq, Sk, H, Hkv, D, dtype, kw)
    ref = bo.attention(q, k, v, do, dtype=dtype, **kw)
    gk = dict(kw, q_len=lens(kw.get("q_len")), kv_len=lens(kw.get("kv_len")))
    place = arrange or (lambda name, t: t)
    qd, kd, vd, dod = (place(n, dev(x, dtype)) for n, x in (("q", q), ("k", k), ("v", v), ("do", do)))
    o, lse = pamm.attention(qd, kd, vd, **gk)
    close("o", o, ref["o"], ref["o_tol"])
    close("lse", lse, ref["lse"], ref["lse_tol"])
    if backward:
        grads = pamm.attention_backward(dod, qd, kd, vd, o, lse, **gk)
        for n, t in zip(("dq", "dk", "dv"), grads):
            close(n, t, ref[n], ref[n + "_tol"])
        again = pamm.attention_backward(dod, qd, kd, vd, o, lse, **gk)
        assert all(torch.equal(a, b) for a, b in zip(grads, again)), "not repeatable"
    return ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 32, 40, 64, 72, 96, 104, 128])
def test_head_dims(dtype, D):
    check(2, 70, 70, 4, 2, D, dtype, causal=True)
    check(1, 33, 97, 2, 2, D, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 2), (2, 1), (31, 33), (32, 32), (63, 65), (64, 128), (127, 129),
                                   (129, 127), (257, 300), (1, 700), (5, 260), (200, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(dtype, Sq, Sk, causal):
    # with more queries than keys the first causal rows see nothing
    check(1, Sq, Sk, 2, 1, 64, dtype, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (8, 1), (40, 1), (5, 5)])
def test_shared_heads(dtype, H, Hkv):
    check(2, 50, 50, H, Hkv, 32, dtype, causal=True)
    check(2, 1, 90, H, Hkv, 32, dtype, causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 10**6])
def test_windows(dtype, window):
    check(1, 150, 150, 2, 1, 64, dtype, causal=True, window=window)
    check(1, 40, 200, 2, 2, 64, dtype, causal=True, window=window)
    check(1, 1, 200, 2, 2, 64, dtype, causal=True, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_lengths(dtype, causal):
    n = [0, 1, 31, 64, 65, 130]
    check(6, 130, 130, 4, 2, 64, dtype, causal=causal, q_len=n, kv_len=n)
    check(6, 130, 200, 2, 2, 40, dtype, causal=causal, kv_len=[0, 200, 1, 77, 129, 130])
    check(4, 100, 60, 2, 1, 64, dtype, causal=causal, q_len=[0, 3, 100, 50])
    # lengths past the tensors and below zero are clamped
    check(3, 20, 30, 2, 1, 64, dtype, causal=causal, q_len=[-5, 99, 20], kv_len=[30, 2**31 - 1, -2**31])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens_over_caches(dtype):
    for B, Sk, H, Hkv, D in ((1, 130, 12, 12, 64), (3, 1000, 8, 2, 128), (5, 4100, 4, 1, 96), (2, 33, 32, 1, 64)):
        n = [max(1, Sk - 37 * b * b) for b in range(B)]
        check(B, 1, Sk, H, Hkv, D, dtype, causal=True, kv_len=n, backward=False)
    # an empty cache among others, whose keys are split over workgroups
    check(3, 1, 2000, 2, 1, 64, dtype, causal=True, kv_len=[2000, 0, 1], backward=False)
    # a few queries, and a chunk whose keys are split
    check(1, 4, 3000, 8, 1, 64, dtype, causal=True, backward=False)
    check(1, 40, 3000, 2, 2, 64, dtype, causal=True, backward=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(dtype):
    for scale in (0.5, -0.3, 0.0, 1e-4):
        check(1, 40, 50, 2, 1, 64, dtype, scale=scale)
    # rows dominated by one key; the maximum moves far between key blocks
    check(1, 100, 200, 2, 1, 64, dtype, causal=True, scale=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orders_and_strides(dtype):
    def heads_first(name, t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def sequence_first(name, t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def padded(name, t):
        buf = torch.full((t.shape[0], t.shape[1] + 3, t.shape[2] + 1, t.shape[3] + 16), float("nan"), dtype=t.dtype,
                         device="cuda")
        buf[:, 1:-2, 1:, 8:-8] = t
        return buf[:, 1:-2, 1:, 8:-8]

    for f in (heads_first, sequence_first, padded):
        check(2, 70, 90, 4, 2, 64, dtype, causal=True, arrange=f)
        check(2, 1, 90, 4, 2, 40, dtype, causal=True, arrange=f, backward=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_in_a_packed_gradient(dtype):
    rng = np.random.default_rng(3)
    B, S, H, Hkv, D = 2, 45, 4, 2, 64
    qkv, do = values(rng, (B, S, H + 2 * Hkv, D), dtype), values(rng, (B, S, H, D), dtype)
    ref = bo.attention(qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:], do, causal=True, dtype=dtype)
    t = dev(qkv, dtype)
    q, k, v = t.split([H, Hkv, Hkv], dim=2)
    o = torch.empty(B, H, S, D, dtype=DT[dtype], device="cuda").transpose(1, 2)
    lse = torch.empty(B, H, S, device="cuda")
    o2, lse2 = pamm.attention(q, k, v, causal=True, o=o, lse=lse)
    assert o2 is o and lse2 is lse
    grad = torch.full_like(t, float("nan"))
    dq, dk, dv = grad.split([H, Hkv, Hkv], dim=2)
    pamm.attention_backward(dev(do, dtype), q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        close(n, x, ref[n], ref[n + "_tol"])


def test_broadcast_keys():
    rng = np.random.default_rng(4)
    q, do = values(rng, (3, 40, 4, 64), "f32"), values(rng, (3, 40, 4, 64), "f32")
    k1, v1 = values(rng, (1, 50, 1, 64), "f32"), values(rng, (1, 50, 1, 64), "f32")
    k, v = np.broadcast_to(k1, (3, 50, 4, 64)), np.broadcast_to(v1, (3, 50, 4, 64))
    ref = bo.attention(q, k, v, do)
    kd, vd = dev(k1, "f32").expand(3, 50, 4, 64), dev(v1, "f32").expand(3, 50, 4, 64)
    o, lse = pamm.attention(dev(q, "f32"), kd, vd)
    close("o", o, ref["o"], ref["o_tol"])
    grads = pamm.attention_backward(dev(do, "f32"), dev(q, "f32"), kd, vd, o, lse)
    for n, t in zip(("dq", "dk", "dv"), grads):
        close(n, t, ref[n], ref[n + "_tol"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Sq", [1, 90])
def test_what_lies_past_the_lengths_is_not_read(dtype, Sq):
    rng = np.random.default_rng(5)
    B, Sk, H, Hkv, D = 3, 90, 4, 2, 64
    n = [40, 0, 90]
    q, do = values(rng, (B, Sq, H, D), dtype), values(rng, (B, Sq, H, D), dtype)
    k, v = values(rng, (B, Sk, Hkv, D), dtype), values(rng, (B, Sk, Hkv, D), dtype)
    ref = bo.attention(q, k, v, do, causal=Sq == 1, kv_len=n, dtype=dtype)
    kd, vd = dev(k, dtype), dev(v, dtype)
    for b, x in enumerate(n):
        kd[b, x:] = float("nan")
        vd[b, x:] = float("inf")
    o, lse = pamm.attention(dev(q, dtype), kd, vd, causal=Sq == 1, kv_len=lens(n))
    close("o", o, ref["o"], ref["o_tol"])
    close("lse", lse, ref["lse"], ref["lse_tol"])
    grads = pamm.attention_backward(dev(do, dtype), dev(q, dtype), kd, vd, o, lse, causal=Sq == 1, kv_len=lens(n))
    for name, t in zip(("dq", "dk", "dv"), grads):
        close(name, t, ref[name], ref[name + "_tol"])


def test_gradient_against_differences():
    """Central differences of the 64-bit forward pass along random directions,
    third derivatives of order one: h = 1e-4 leaves ~1e-8 of the derivative."""
    rng = np.random.default_rng(6)
    B, S, H, Hkv, D, h = 1, 37, 4, 2, 32, 1e-4
    kw = {"causal": True, "window": 20}
    x = {"q": values(rng, (B, S, H, D), "f32"), "k": values(rng, (B, S, Hkv, D), "f32"),
         "v": values(rng, (B, S, Hkv, D), "f32")}
    do = values(rng, (B, S, H, D), "f32")
    d = {n: dev(t, "f32") for n, t in x.items()}
    o, lse = pamm.attention(d["q"], d["k"], d["v"], **kw)
    grads = dict(zip("qkv", pamm.attention_backward(dev(do, "f32"), d["q"], d["k"], d["v"], o, lse, **kw)))
    ref = bo.attention(x["q"], x["k"], x["v"], do, **kw)

    def loss(**change):
        y = {**x, **change}
        return (bo.attention(y["q"], y["k"], y["v"], **kw)["o"] * do).sum()

    for n in "qkv":
        for _ in range(3):
            way = rng.standard_normal(x[n].shape)
            diff = (loss(**{n: x[n] + h * way}) - loss(**{n: x[n] - h * way})) / (2 * h)
            got = (host(grads[n]) * way).sum()
            tol = (ref[f"d{n}_tol"] * np.abs(way)).sum() + 1e-6 * np.linalg.norm(host(grads[n])) * np.linalg.norm(way)
            assert abs(got - diff) <= tol, (n, got, diff, tol)


def test_other_stream_and_workspace():
    rng = np.random.default_rng(7)
    q, k, v = (dev(values(rng, s, "bf16"), "bf16") for s in ((2, 1, 4, 64), (2, 2000, 2, 64), (2, 2000, 2, 64)))
    o, lse = pamm.attention(q, k, v)
    need = pamm.attention_workspace_size(q, k)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = pamm.attention(q, k, v, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    with torch.cuda.stream(side):
        o3, _ = pamm.attention(q, k, v, workspace=ws)
    side.synchronize()
    assert torch.equal(o, o3)


def test_long_cache_past_32_bit_offsets():
    """Keys whose byte offsets pass 2^32: the last ones decide the result."""
    Sk, Hkv, D = 2_200_000, 8, 128  # 4.5 GB each
    k = torch.zeros(1, Sk, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.ones(1, 1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    k[0, -1] = 8.0  # score 8 * 128 / sqrt(128): all of the weight
    v[0, -1] = torch.arange(D, device="cuda").to(torch.bfloat16)
    o, _ = pamm.attention(q, k, v, causal=True)
    assert torch.equal(o[0, 0], v[0, -1])
    q40 = q.expand(1, 40, Hkv, D)
    o, _ = pamm.attention(q40, k, v)
    assert torch.equal(o[0, 39], v[0, -1]) and torch.equal(o[0, 0], v[0, -1])


def test_refusals():
    q = torch.zeros(2, 8, 4, 64, device="cuda")
    k = torch.zeros(2, 8, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        pamm.attention(q, torch.zeros(2, 8, 3, 64, device="cuda"), torch.zeros(2, 8, 3, 64, device="cuda"))
    with pytest.raises(ValueError):
        pamm.attention(q, k, k[:, :7])
    with pytest.raises(ValueError):
        pamm.attention(q[0], k, k)
    with pytest.raises(TypeError):
        pamm.attention(q, k.bfloat16(), k.bfloat16())
    with pytest.raises(TypeError):
        pamm.attention(q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        pamm.attention(q, k.cpu(), k.cpu())
    with pytest.raises(ValueError):
        pamm.attention(q.transpose(2, 3), k, k)
    with pytest.raises(TypeError):
        pamm.attention(q, k, k, kv_len=torch.tensor([8, 8], device="cuda"))
    with pytest.raises(ValueError):
        pamm.attention(q, k, k, kv_len=torch.tensor([8], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pamm.attention(q, k, k, o=torch.zeros(2, 1, 4, 64, device="cuda").expand(2, 8, 4, 64))
    for kw in ({"window": 4}, {"scale": float("nan")}, {"window": -1, "causal": True}):
        with pytest.raises(pamm.PammError):
            pamm.attention(q, k, k, **kw)
    big = torch.zeros(1, 4, 1, 136, device="cuda")
    with pytest.raises(pamm.PammError):
        pamm.attention(big, big, big)
    odd = torch.zeros(1, 4, 1, 64, device="cuda")[..., :6]
    with pytest.raises(pamm.PammError):
        pamm.attention(odd, odd, odd)
    o, lse = pamm.attention(q, k, k)
    with pytest.raises(ValueError):
        pamm.attention_backward(o[:, :4], q, k, k, o, lse)
    with pytest.raises(ValueError):
        pamm.attention_backward(o, q, k, k, o, lse[:, :, :4])
    long = k.repeat(1, 300, 1, 1)
    with pytest.raises(ValueError):
        pamm.attention(q[:, :1], long, long, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))


def test_empty_sizes():
    for B, Sq, Sk in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        q, k = torch.ones(B, Sq, 4, 64, device="cuda"), torch.ones(B, Sk, 2, 64, device="cuda")
        o, lse = pamm.attention(q, k, k)
        assert not o.any() and bool((lse == -float("inf")).all())
        dq, dk, dv = pamm.attention_backward(torch.ones_like(o), q, k, k, o, lse)
        assert not dq.any() and not dk.any() and not dv.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Sq,Sk,D,window", [(150, 150, 64, 0), (150, 150, 128, 40), (100, 230, 40, 0), (9, 200, 96, 0),
                                            (9, 200, 64, 5), (40, 3000, 64, 0)])
def test_hidden_infinities_and_nans(dtype, Sq, Sk, D, window):
    """Something not finite in a key or query reaches what sees it, and nothing else."""
    rng = np.random.default_rng(8)
    H, Hkv = 4, 2
    kw = {"causal": True, "window": window}
    x = {n: values(rng, s, dtype) for n, s in (("q", (1, Sq, H, D)), ("k", (1, Sk, Hkv, D)), ("v", (1, Sk, Hkv, D)),
                                               ("do", (1, Sq, H, D)))}
    ref = bo.attention(x["q"], x["k"], x["v"], x["do"], dtype=dtype, **kw)
    m = bo.visible(Sq, Sk, Sq, Sk, True, window)

    def run(changes):
        d = {n: dev(t, dtype) for n, t in x.items()}
        for name, at, head, value in changes:
            d[name][0, at, head, D // 2] = value
        o, lse = pamm.attention(d["q"], d["k"], d["v"], **kw)
        return dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *pamm.attention_backward(
            d["do"], d["q"], d["k"], d["v"], o, lse, **kw))))

    def clean(got, name, where, heads):
        a, b = host(got[name])[0][where][:, heads], ref[name][0][where][:, heads]
        close(name, a, b, ref[name + "_tol"][0][where][:, heads])

    nan, inf = float("nan"), float("inf")
    for j0 in sorted({0, Sk - Sq // 2 - 1, Sk - 1}):
        hit = m[:, j0]
        touched = m[hit].any(0)
        for changes in ([("v", j0, 0, inf)], [("v", j0, 0, -inf)], [("v", j0, 0, nan)], [("k", j0, 0, nan), ("v", j0, 0, nan)]):
            say("hidden key", j0, changes)
            got = run(changes)
            every, group = slice(None), slice(0, H // Hkv)  # the other heads are not touched at all
            rest = slice(H // Hkv, H)
            for n in ("o", "dq"):
                clean(got, n, slice(None), rest)
                clean(got, n, ~hit, group)
            for n in ("dk", "dv"):
                clean(got, n, slice(None), slice(1, Hkv))
            for n in ("dk", "dv"):
                clean(got, n, ~touched, slice(0, 1))
            seen = host(got["o"])[0][hit][:, group, D // 2]
            want = changes[0][3] if len(changes) == 1 else nan
            assert np.array_equal(seen, np.full(seen.shape, want), equal_nan=True), (j0, changes)
            if len(changes) == 1:  # only that column of the output
                other = np.arange(D) != D // 2
                close("o", host(got["o"])[0][hit][:, group][..., other], ref["o"][0][hit][:, group][..., other],
                      ref["o_tol"][0][hit][:, group][..., other])
                close("lse", got["lse"], ref["lse"], ref["lse_tol"])
    for i0 in sorted({0, Sq // 3, Sq - 1}):
        others = np.arange(Sq) != i0
        for changes in ([("do", i0, 1, nan)], [("do", i0, 1, inf)], [("q", i0, 1, nan)]):
            say("hidden query", i0, changes)
            got = run(changes)
            for n in ("o", "dq"):
                clean(got, n, others, slice(None))
            for n in ("dk", "dv"):
                clean(got, n, ~m[i0], slice(None))
                clean(got, n, slice(None), slice(1, Hkv))
            keys = m[i0]
            bad = host(got["dv"])[0][keys][:, 0, D // 2]
            assert not np.isfinite(bad).any(), (i0, changes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Sq", [5, 70])
def test_rows_past_the_lengths_are_zero_beside_nans(dtype, causal, Sq):
    rng = np.random.default_rng(9)
    B, Sk, H, Hkv, D, Lq, Lk = 1, 80, 4, 2, 64, Sq - 3, 45
    d = {n: dev(values(rng, s, dtype), dtype) for n, s in (("q", (B, Sq, H, D)), ("k", (B, Sk, Hkv, D)),
                                                           ("v", (B, Sk, Hkv, D)), ("do", (B, Sq, H, D)))}
    for n, at in (("q", 1), ("k", 3), ("v", 4), ("do", 0)):
        d[n][:, at] = float("nan")
    kw = {"causal": causal, "q_len": lens([Lq]), "kv_len": lens([Lk])}
    o, lse = pamm.attention(d["q"], d["k"], d["v"], **kw)
    dq, dk, dv = pamm.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, **kw)
    if not causal or 1 + Lk - Lq >= 4:  # query 1 sees the keys that hold NaNs
        assert torch.isnan(o[:, 1]).all()
    assert (o[:, Lq:] == 0).all() and (dq[:, Lq:] == 0).all() and bool((lse[:, :, Lq:] == -float("inf")).all())
    assert (dk[:, Lk:] == 0).all() and (dv[:, Lk:] == 0).all()
