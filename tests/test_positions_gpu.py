"""GPU: the rotation of queries and keys, their norm and its gradients against
the plain 64-bit definitions (tests/position_oracle.py, which also derives the
bounds), at the sizes, layouts and positions where they can go wrong."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import position_oracle as po
from test_attention_gpu import DT, close, dev, host, say, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BOTH = pytest.mark.parametrize("dtype", ["bf16", "f32"])
KINDS = pytest.mark.parametrize("interleaved", [False, True])


def freqs(rot, device="cuda"):
    return pamm.rotary_frequencies(rot, device=device)[0]


def where(rng, B, S, kind, far=0):
    """positions as the call takes them, and [B, S] numbers"""
    p = np.broadcast_to(np.arange(S), (B, S)).astype(np.int64)
    kw = {}
    if kind in ("each", "each32", "both"):
        p = rng.integers(-50, 50, (B, S)) + far
        kw["positions"] = torch.tensor(p, dtype=torch.int32 if kind == "each32" else torch.int64, device="cuda")
    if kind == "row":
        p = np.broadcast_to(rng.integers(0, 500, S) + far, (B, S))
        kw["positions"] = torch.tensor(p[0].copy(), device="cuda")
    if kind in ("offset", "both"):
        o = rng.integers(0, 1000, B) + (far if kind == "offset" else 0)
        kw["offset"] = torch.tensor(o, dtype=torch.int32, device="cuda")
        p = p + o[:, None]
    return kw, p


def check(B, S, H, Hkv, D, rot, dtype, *, interleaved=False, magnitude=1.0, eps=1e-6, kind="none", far=0, seed=0,
          place=lambda n, t: t, plain=True):
    say("positions", B, S, H, Hkv, D, rot, dtype, interleaved, kind, far)
    rng = np.random.default_rng(seed)
    q, k = values(rng, (B, S, H, D), dtype, 2.0), values(rng, (B, S, Hkv, D), dtype)
    dq, dk = values(rng, (B, S, H, D), dtype), values(rng, (B, S, Hkv, D), dtype)
    wq, wk = (host(dev(1 + 0.2 * rng.standard_normal(D), dtype)) for _ in range(2))
    f = freqs(rot)
    kw, pos = where(rng, B, S, kind, far)
    both = dict(interleaved=interleaved, magnitude=magnitude)
    qd, kd, dqd, dkd = (place(n, dev(t, dtype)) for n, t in (("q", q), ("k", k), ("dq", dq), ("dk", dk)))
    if plain:
        for x, xd in ((q, qd), (k, kd)):
            for inverse in (False, True):
                y, tol = po.rotary(x, pos, host(f), dtype=dtype, inverse=inverse, **both)
                close("rotary", pamm.rotary(xd, f, inverse=inverse, **both, **kw), y, tol)
    args = (qd, kd, dev(wq, dtype), dev(wk, dtype), f)
    qo, ko = pamm.qk_norm_rotary(*args, eps=eps, **both, **kw)
    grads = pamm.qk_norm_rotary_backward(dqd, dkd, *args, eps=eps, **both, **kw)
    again = pamm.qk_norm_rotary_backward(dqd, dkd, *args, eps=eps, **both, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)), "not repeatable"
    for n, x, w, dy, y, dx, dw in (("q", q, wq, dq, qo, grads[0], grads[2]), ("k", k, wk, dk, ko, grads[1], grads[3])):
        ref = po.norm_rotary(x, w, pos, host(f), eps=eps, dy=dy, dtype=dtype, **both)
        close(n, y, ref["y"], ref["y_tol"])
        close("d" + n, dx, ref["dx"], ref["dx_tol"])
        close("dw" + n, dw, ref["dw"], ref["dw_tol"])


@BOTH
@KINDS
@pytest.mark.parametrize("D,rot", [(8, 8), (8, 2), (16, 16), (24, 24), (32, 16), (40, 20), (40, 40), (64, 64), (64, 30),
                                   (72, 18), (80, 80), (96, 48), (104, 104), (112, 2), (128, 128), (128, 64), (128, 126),
                                   (64, 0)])
def test_head_dims(dtype, interleaved, D, rot):
    if rot:
        check(2, 7, 3, 2, D, rot, dtype, interleaved=interleaved, magnitude=1.25, kind="each")
    else:
        check(2, 7, 3, 2, D, rot, dtype, interleaved=interleaved, kind="each")


@BOTH
@pytest.mark.parametrize("B,S,H,Hkv", [(1, 1, 1, 1), (1, 1, 32, 8), (64, 1, 12, 12), (3, 333, 6, 2), (1, 2049, 4, 1),
                                       (5, 17, 1, 1), (2, 700, 33, 7), (1, 5000, 2, 2), (1, 3, 257, 5)])
def test_sizes(dtype, B, S, H, Hkv):
    check(B, S, H, Hkv, 64, 64, dtype, kind="offset", plain=S < 1000)


@BOTH
def test_many_tokens(dtype):
    """More tokens than the backward pass has workgroups at a time, so that each loops."""
    check(1, 6000, 2, 1, 16, 16, dtype, kind="both", plain=False)
    check(2, 9001, 1, 1, 8, 4, dtype, interleaved=True, plain=False)


@BOTH
@KINDS
@pytest.mark.parametrize("kind", ["none", "offset", "each", "each32", "row", "both"])
@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 31) - 2000])
def test_positions(dtype, interleaved, kind, far):
    check(2, 9, 2, 1, 32, 32, dtype, interleaved=interleaved, kind=kind, far=far)


def test_strided_positions():
    f, x = freqs(16), torch.randn(2, 6, 2, 16, device="cuda")
    p = torch.randint(0, 1000, (6, 2, 3), device="cuda")
    assert torch.equal(pamm.rotary(x, f, positions=p[:, :, 1].T), pamm.rotary(x, f, positions=p[:, :, 1].T.contiguous()))
    assert torch.equal(pamm.rotary(x, f, positions=p[:, 0, 0]), pamm.rotary(x, f, positions=p[:, 0, 0].contiguous()))
    row = torch.arange(6, device="cuda")
    assert torch.equal(pamm.rotary(x, f, positions=row[None].expand(2, -1)), pamm.rotary(x, f))


@BOTH
def test_layouts(dtype):
    """Any order of the outer dimensions, slices of a packed projection output, broadcast inputs."""
    perms = {"q": (2, 0, 1, 3), "k": (1, 2, 0, 3), "dq": (0, 2, 1, 3), "dk": (2, 1, 0, 3)}

    def place(name, t):
        p = perms[name]
        return t.permute(p).contiguous().permute([p.index(i) for i in range(4)])

    check(2, 19, 4, 2, 64, 32, dtype, place=place)
    packed = torch.randn(2, 19, 8, 64, device="cuda").to(DT[dtype])
    f, w = freqs(64), torch.ones(64, device="cuda", dtype=DT[dtype])
    q, k, _ = packed.split([4, 2, 2], dim=2)
    a, b = pamm.qk_norm_rotary(q, k, w, w, f)
    c, d = pamm.qk_norm_rotary(q.contiguous(), k.contiguous(), w, w, f)
    assert torch.equal(a, c) and torch.equal(b, d)
    one = torch.randn(1, 19, 1, 64, device="cuda").to(DT[dtype])
    assert torch.equal(pamm.rotary(one.expand(3, 19, 5, 64), f), pamm.rotary(one.expand(3, 19, 5, 64).contiguous(), f))


@BOTH
@KINDS
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (40, 20), (72, 10)])
def test_in_place(dtype, interleaved, D, rot):
    g = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randn(2, 50, 7, D, generator=g, device="cuda").to(DT[dtype])
    f, w = freqs(rot), torch.full((D,), 1.5, device="cuda", dtype=DT[dtype])
    q, k, v = packed.split([4, 2, 1], dim=2)
    want, keep = pamm.rotary(packed[:, :, :6], f, interleaved=interleaved), v.clone()
    wq, wk = pamm.qk_norm_rotary(q, k, w, w, f, interleaved=interleaved)
    mine = packed.clone()
    assert pamm.rotary(mine[:, :, :6], f, interleaved=interleaved, out=mine[:, :, :6]).data_ptr() == mine.data_ptr()
    assert torch.equal(mine[:, :, :6], want) and torch.equal(mine[:, :, 6:], keep)
    mine = packed.clone()
    mq, mk, mv = mine.split([4, 2, 1], dim=2)
    pamm.qk_norm_rotary(mq, mk, w, w, f, interleaved=interleaved, q_out=mq, k_out=mk)
    assert torch.equal(mq, wq) and torch.equal(mk, wk) and torch.equal(mv, keep)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    a = pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, interleaved=interleaved)
    b = pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, interleaved=interleaved, dq_out=dq, dk_out=dk)
    assert b[0].data_ptr() == dq.data_ptr() and all(torch.equal(x, y) for x, y in zip(a, b))


@BOTH
@KINDS
def test_the_inverse_turns_back(dtype, interleaved):
    """Two rotations of 32-bit rows cancel to their errors; what is not rotated is copied bit by bit."""
    x = torch.randn(2, 100, 3, 48, device="cuda").to(DT[dtype])
    f = freqs(32)
    y = pamm.rotary(x, f, interleaved=interleaved)
    assert torch.equal(y[..., 32:], x[..., 32:]) and torch.equal(y[:, 0], x[:, 0])
    z = pamm.rotary(y, f, interleaved=interleaved, inverse=True)
    # each rotation rounds twice the size of a pair's elements at most
    tol = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -20) * 2 * x.abs().max()
    assert (z.float() - x.float()).abs().max() <= tol


@BOTH
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 64, True), (40, 20, False)])
def test_what_is_not_finite_stays_in_its_row(dtype, D, rot, interleaved):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(2, 40, 5, D, generator=g, device="cuda").to(DT[dtype])
    w, f = torch.ones(D, device="cuda", dtype=DT[dtype]), freqs(rot)
    dy = torch.randn(2, 40, 5, D, generator=g, device="cuda").to(DT[dtype])
    bad = x.clone()
    bad[1, 7, 2, 3], bad[0, 3, 4, 9], bad[0, 39, 0, 0] = float("nan"), float("inf"), 3e38
    hit = torch.zeros(2, 40, 5, dtype=torch.bool, device="cuda")
    hit[1, 7, 2] = hit[0, 3, 4] = hit[0, 39, 0] = True
    for fn in (lambda t: pamm.rotary(t, f, interleaved=interleaved),
               lambda t: pamm.qk_norm_rotary(t, x, w, w, f, interleaved=interleaved)[0],
               lambda t: pamm.qk_norm_rotary_backward(dy, dy, t, x, w, w, f, interleaved=interleaved)[0]):
        assert torch.equal(fn(bad)[~hit], fn(x)[~hit])
    y = pamm.qk_norm_rotary(bad, x, w, w, f, interleaved=interleaved)[0]
    assert torch.isnan(y[1, 7, 2]).all() and not y[0, 39, 0].any()
    pos = torch.zeros(2, 40, dtype=torch.int64, device="cuda")
    nan = torch.full((rot // 2,), float("nan"), dtype=torch.float64, device="cuda")
    assert torch.isnan(pamm.rotary(x, nan, interleaved=interleaved)[..., :rot]).all()
    assert torch.equal(pamm.rotary(x, f, positions=pos, interleaved=interleaved), x)


@BOTH
@KINDS
@pytest.mark.parametrize("D,rot", [(48, 32), (64, 30), (16, 2), (128, 64), (40, 8)])
def test_elements_that_are_not_rotated_stand_alone(dtype, interleaved, D, rot):
    """They are copied one by one: none is reached by another's infinity, and a zero keeps its sign."""
    say("not rotated", dtype, interleaved, D, rot)
    f, w = freqs(rot), torch.ones(D, device="cuda", dtype=DT[dtype])
    x = torch.randn(2, 5, 3, D, device="cuda").to(DT[dtype])
    bad = x.clone()
    bad[..., rot + 1], bad[..., D - 1], bad[..., D - 2] = -0.0, float("inf"), -1.0
    bad[0, 1, :, rot] = float("nan")
    y, clean = (pamm.rotary(t, f, interleaved=interleaved) for t in (bad, x))
    assert torch.equal(y[..., :rot], clean[..., :rot])
    assert torch.equal(y[..., rot:].nan_to_num(7.0, 8.0), bad[..., rot:].nan_to_num(7.0, 8.0))
    assert torch.signbit(y[..., rot + 1]).all()
    # a norm's row with one infinity: NaN in its place, zeros elsewhere
    one = x.clone()
    one[..., D - 1] = float("inf")
    y = pamm.qk_norm_rotary(one, x, w, w, f, interleaved=interleaved)[0]
    assert torch.isnan(y[..., D - 1]).all() and not y[..., :D - 1].any()
    # a gradient that is not finite reaches its own element of the weight's
    dy = torch.randn_like(x)
    dy[1, 2, 0, D - 1] = float("inf")
    dw = pamm.qk_norm_rotary_backward(dy, x, x, x, w, w, f, interleaved=interleaved)[2]
    assert torch.isfinite(dw[:D - 1]).all() and not torch.isfinite(dw[D - 1])


def test_zero_rows_and_eps():
    x, w, f = torch.zeros(1, 4, 2, 32, device="cuda"), torch.ones(32, device="cuda"), freqs(32)
    y, _ = pamm.qk_norm_rotary(x, x, w, w, f)
    dx, _, dw, _ = pamm.qk_norm_rotary_backward(torch.ones_like(x), x, x, x, w, w, f)
    assert not y.any() and not dw.any() and torch.isfinite(dx).all()
    check(1, 4, 2, 2, 32, 32, "f32", eps=0.5)


def test_gradients_against_differences():
    """The gradient of sum(dy y) by differences of the 32-bit kernel: with a step of 2^-6, the
    difference's own error is its third derivative's (1e-4 of values of size 1) and y's 2^-22 / 2^-6."""
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k, dq, dk, wq, wk, f = r(1, 3, 2, 8), r(1, 3, 1, 8), r(1, 3, 2, 8), r(1, 3, 1, 8), r(8), r(8), freqs(6)
    kw = dict(eps=0.1, magnitude=1.1, positions=torch.tensor([3, 70, 5], device="cuda"))

    def loss(*a):
        x, y = pamm.qk_norm_rotary(*a, f, **kw)
        return ((x.double() * dq).sum() + (y.double() * dk).sum()).item()

    args = [q, k, wq, wk]
    grads = pamm.qk_norm_rotary_backward(dq, dk, q, k, wq, wk, f, **kw)
    for n, (t, got) in enumerate(zip(args, grads)):
        for i in range(t.numel()):
            sides = []
            for step in (2.0 ** -6, -2.0 ** -6):
                moved = t.clone()
                moved.view(-1)[i] += step
                sides.append(loss(*(moved if j == n else a for j, a in enumerate(args))))
            want = (sides[0] - sides[1]) / 2.0 ** -5
            assert abs(got.reshape(-1)[i].item() - want) < 5e-3 * max(1.0, abs(want)), (n, i)


def test_empty_calls():
    f, w = freqs(16), torch.ones(16, device="cuda")
    for shape in ((0, 5, 2, 16), (3, 0, 2, 16)):
        x = torch.empty(shape, device="cuda")
        assert pamm.rotary(x, f).shape == shape
        assert pamm.qk_norm_rotary(x, x, w, w, f)[1].shape == shape
        _, _, a, b = pamm.qk_norm_rotary_backward(x, x, x, x, w, w, f)
        assert not a.any() and not b.any() and a.shape == b.shape == (16,)


def test_workspace_and_stream():
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    q, k, dq, dk, w, f = r(2, 300, 4, 64), r(2, 300, 2, 64), r(2, 300, 4, 64), r(2, 300, 2, 64), r(64), freqs(64)
    ws = torch.empty(pamm.qk_norm_rotary_backward_workspace_size(q, k), dtype=torch.uint8, device="cuda")
    want = pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, workspace=ws[:64])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = [lambda s: pamm.qk_norm_rotary_backward(dq, dk, q, k, w, w, f, stream=s),
             lambda s: pamm.qk_norm_rotary(q, k, w, w, f, stream=s), lambda s: (pamm.rotary(q, f, stream=s),)]
    for i, call in enumerate(calls):
        ref = want if i == 0 else call(None)
        got = call(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@BOTH
@KINDS
@pytest.mark.parametrize("B,S,H,Hkv", [(1, 1, 4, 2), (2, 700, 8, 1), (3, 5, 2, 9)])
def test_queries_and_keys_without_weights_in_one_call(dtype, interleaved, B, S, H, Hkv):
    """The C call takes both without a norm, too."""
    from activation_compression_pamm_amd import position_ops as ops
    from activation_compression_pamm_amd.block_ops import _code, _heads_tensor

    q, k = (torch.randn(B, S, h, 64, device="cuda").to(DT[dtype]) for h in (H, Hkv))
    f, qo, ko = freqs(32), torch.empty_like(q), torch.empty_like(k)
    h = [x for t in (q, k, qo, ko) for x in _heads_tensor("", "", t)]
    p = ops._pack_rotary(_code("", q), int(interleaved), 0, 0, B, S, H, Hkv, 64, 32, 1.0, 0.0, f.data_ptr(), 0, 0, 0, 0, 0,
                         0, *h)
    assert ops._lib().pamm_rotary(p, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(qo, pamm.rotary(q, f, interleaved=interleaved))
    assert torch.equal(ko, pamm.rotary(k, f, interleaved=interleaved))


def test_far_rows():
    """Byte offsets past 2^32 between tokens and heads."""
    big = torch.empty(3 * (1 << 30) + (1 << 10), dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 2, 2, 64), (1 << 29, 1 << 28, (1 << 31) + (1 << 27) + 64, 1), 0)
    x.copy_(torch.randn(2, 2, 2, 64, device="cuda"))
    f = freqs(64)
    assert torch.equal(pamm.rotary(x, f, out=torch.empty(2, 2, 2, 64, device="cuda", dtype=torch.bfloat16)),
                       pamm.rotary(x.contiguous(), f))
