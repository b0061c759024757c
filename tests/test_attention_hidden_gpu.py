"""GPU: what a mask hides does not come through, and what it shows touches
nothing else, for single queries (shared heads, split keys, windows) and in the
second pass over marked work, against tests/block_oracle.py."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import close, dev, host, lens, say, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def single(dtype, H, Hkv, Sk, D=64, B=2, **kw):
    """One query a sequence: the inputs and the exact results of finite data."""
    rng = np.random.default_rng(12)
    x = {n: values(rng, s, dtype) for n, s in (("q", (B, 1, H, D)), ("k", (B, Sk, Hkv, D)), ("v", (B, Sk, Hkv, D)))}
    return x, bo.attention(x["q"], x["k"], x["v"], dtype=dtype, **kw)


def call(d, **kw):
    return pamm.attention(d["q"], d["k"], d["v"], **dict(kw, kv_len=lens(kw.get("kv_len"))))


def same(got, ref, pick=slice(None), columns=slice(None)):
    """o of the heads `pick` in `columns` and lse of those heads."""
    o, lse = got
    close("o", host(o)[:, :, pick][..., columns], ref["o"][:, :, pick][..., columns],
          ref["o_tol"][:, :, pick][..., columns])
    close("lse", host(lse)[:, pick], ref["lse"][:, pick], ref["lse_tol"][:, pick])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (32, 1), (40, 1), (80, 2)])
@pytest.mark.parametrize("Sk", [300, 2000])
def test_one_query_of_many_heads(dtype, H, Hkv, Sk):
    """What is not finite in a head's query or in one column of V stays there."""
    say("one query", dtype, H, Hkv, Sk)
    kw = {"causal": True}
    x, ref = single(dtype, H, Hkv, Sk, **kw)
    d = {n: dev(t, dtype) for n, t in x.items()}
    d["q"][:, 0, 3, 5] = float("nan")
    got = call(d, **kw)
    same(got, ref, np.arange(H) != 3)
    assert torch.isnan(got[0][:, 0, 3]).all() and torch.isnan(got[1][:, 3]).all()
    for value in (float("inf"), float("nan")):
        d = {n: dev(t, dtype) for n, t in x.items()}
        d["v"][:, Sk - 9, 0, 7] = value
        got = call(d, **kw)
        G = H // Hkv
        same(got, ref, slice(None), np.arange(64) != 7)
        same(got, ref, slice(G, None))
        seen = host(got[0])[:, 0, :G, 7]
        assert np.array_equal(seen, np.full(seen.shape, value), equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (40, 1)])
def test_gradients_of_one_query(dtype, H, Hkv):
    """A NaN in one head's dout and an infinity in a key that the query sees."""
    say("gradients of one query", dtype, H, Hkv)
    B, Sk, D, G = 2, 150, 64, H // Hkv
    x, _ = single(dtype, H, Hkv, Sk)
    x["do"] = values(np.random.default_rng(13), (B, 1, H, D), dtype)
    ref = bo.attention(x["q"], x["k"], x["v"], x["do"], causal=True, dtype=dtype)
    d = {n: dev(t, dtype) for n, t in x.items()}
    o, lse = call(d, causal=True)
    d["do"][:, 0, 3, 5] = float("nan")
    dq, dk, dv = pamm.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, causal=True)
    other = np.arange(H) != 3
    close("dq", host(dq)[:, :, other], ref["dq"][:, :, other], ref["dq_tol"][:, :, other])
    hit = 3 // G
    for n, t in (("dk", dk), ("dv", dv)):
        rest = np.arange(Hkv) != hit
        close(n, host(t)[:, :, rest], ref[n][:, :, rest], ref[n + "_tol"][:, :, rest])
    assert torch.isnan(dv[:, :, hit, 5]).all() and torch.isnan(dq[:, 0, 3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (40, 1)])
@pytest.mark.parametrize("Sk,window", [(200, 5), (300, 33), (300, 64), (2000, 37), (3000, 1500)])
def test_one_query_with_a_window(dtype, H, Hkv, Sk, window):
    """Expired keys, in the window's first block and before it, hold anything."""
    say("window", dtype, H, Hkv, Sk, window)
    n = [Sk, Sk - 50]
    kw = {"causal": True, "window": window, "kv_len": n}
    x, ref = single(dtype, H, Hkv, Sk, **kw)
    for value in (float("nan"), float("inf"), float("-inf")):
        for back in (1, 2, 40):  # so many keys before the window
            d = {n: dev(t, dtype) for n, t in x.items()}
            for b in range(2):
                at = max(n[b] - window - back, 0)
                d["v"][b, at, :, 7] = value
                d["k"][b, at, :, 9] = value
                d["v"][b, n[b]:], d["k"][b, n[b]:] = value, value
            same(call(d, **kw), ref)
    # beside that, what the window shows is taken up
    d["v"][:, n[1] - 2, 0, 7] = float("inf")
    got = call(d, **kw)
    same(got, ref, slice(None), np.arange(64) != 7)
    first = host(got[0])[1, 0, :H // Hkv, 7]
    assert np.array_equal(first, np.full(first.shape, np.inf)) if window > 1 else np.isfinite(first).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_one_query_with_a_window(dtype):
    say("gradients of one query with a window", dtype)
    H, Hkv, Sk, kw = 8, 2, 150, {"causal": True, "window": 21}
    x, _ = single(dtype, H, Hkv, Sk)
    x["do"] = values(np.random.default_rng(14), (2, 1, H, 64), dtype)
    ref = bo.attention(x["q"], x["k"], x["v"], x["do"], dtype=dtype, **kw)
    d = {n: dev(t, dtype) for n, t in x.items()}
    d["k"][:, Sk - 22, :, 3], d["v"][:, Sk - 23, :, 4] = float("nan"), float("inf")
    o, lse = call(d, **kw)
    for n, t in zip(("o", "lse", "dq", "dk", "dv"),
                    (o, lse, *pamm.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, **kw))):
        close(n, t, ref[n], ref[n + "_tol"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,S,H,Hkv,D,window", [(1, 500, 4, 4, 64, 8), (1, 500, 4, 2, 128, 16), (2, 200, 4, 2, 64, 0),
                                                (1, 300, 2, 2, 96, 50), (16, 1030, 4, 4, 32, 0)])
def test_the_second_pass_computes_what_the_first_does(dtype, B, S, H, Hkv, D, window):
    """With o and lse the same, gradients that nothing reaches of what is not
    finite have the same bits as without it, whether dq and dk/dv run in one
    launch or (short windows in bf16, many items) in two."""
    say("second pass", dtype, B, S, H, Hkv, D, window)
    rng = np.random.default_rng(15)
    kw = {"causal": True, "window": window}
    d = {n: dev(values(rng, s, dtype), dtype) for n, s in (("q", (B, S, H, D)), ("k", (B, S, Hkv, D)), ("v", (B, S, Hkv, D)),
                                                           ("do", (B, S, H, D)))}
    o, lse = pamm.attention(d["q"], d["k"], d["v"], **kw)

    def gradients(**change):
        c = {**d, **change}
        return pamm.attention_backward(c["do"], c["q"], c["k"], c["v"], o, lse, **kw)

    want = gradients()
    m = torch.from_numpy(bo.visible(S, S, S, S, True, window)).cuda()
    for name in ("k", "v", "q", "do"):
        for at in (S // 2, S - 5):
            t = d[name].clone()
            t[0, at, 0, 3] = float("nan")
            dq, dk, dv = gradients(**{name: t})
            rows = ~m[:, at] if name in "kv" else torch.arange(S, device="cuda") != at
            keys = ~(m[~rows].any(0))
            assert torch.equal(dq[0][rows], want[0][0][rows]), (name, at)
            assert torch.equal(dk[0][keys], want[1][0][keys]) and torch.equal(dv[0][keys], want[2][0][keys]), (name, at)
            assert all(torch.equal(x[1:], y[1:]) for x, y in zip((dq, dk, dv), want))
            assert not torch.isfinite(dk if name in ("q", "do") else dq).all()
