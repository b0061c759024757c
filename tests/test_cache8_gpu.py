"""GPU: a cache in 8 bits, and attention over it, against the plain 64-bit
definitions (tests/cache_oracle.py, tests/block_oracle.py), at the lengths,
chunks and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
import cache_oracle as co
from test_attention_gpu import DT, close, dev, host, lens, say, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BOTH = pytest.mark.parametrize("dtype", ["bf16", "f32"])
MARK = 0x5A  # bytes that no call may touch


def filled(B, room, H, D, block, dtype):
    c = pamm.CacheFP8.empty(B, room, H, D, block=block, dtype=DT[dtype])
    for t in c:
        t.transpose(1, 2).view(torch.uint8).fill_(MARK)
    return c


def raw(t):
    """bytes [B, rows, H, D of them]"""
    return t.transpose(1, 2).view(torch.uint8).transpose(1, 2).cpu().numpy()


def marked(t):
    return (raw(t) == MARK).all()


def holds(c, name, tokens, dtype):
    """The cache's `name` is what the tokens (a list of [L, H, D]) make, and nothing else was written."""
    kind = {"k": (c.k, c.k_scale, c.k_tail), "v": (c.v, c.v_scale, c.v_tail)}[name]
    eight, scale, tail = kind
    block = tail.shape[1]
    got, gs, gt = host(eight.float()), host(scale), host(tail.float())
    for b, x in enumerate(tokens):
        q, s = co.blocks(x, block)
        S, n = q.shape[0], len(x) - q.shape[0]
        same = (got[b, :S] == q) | (np.isnan(got[b, :S]) & np.isnan(q))
        if dtype == "f32":
            with np.errstate(invalid="ignore"):
                same |= co.near_tie(np.where(np.isfinite(x), x, 0.0), block) & (np.abs(got[b, :S] - q) <= np.abs(q) / 8 + 2.0 ** -9)
        assert same.all(), (name, b, np.argwhere(~same)[0], got[b, :S][~same][0], q[~same][0])
        assert (np.abs(gs[b, :S // block] - s) <= bo.U * s).all(), (name, b, "scale")
        assert np.array_equal(gt[b, :n], x[S:], equal_nan=True), (name, b, "tail")
        assert marked(eight[b:b + 1, S:]) and marked(scale[b:b + 1, S // block:, :, None]), (name, b, "behind")
        if len(x) < block:
            assert marked(tail[b:b + 1, n:]), (name, b, "tail behind")


def tokens(rng, lengths, H, D, dtype):
    return [values(rng, (n, H, D), dtype) * rng.uniform(0.5, 4, (1, H, 1)) for n in lengths]


def rounded(xs, dtype):
    return [bo.to_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64) for x in xs]


def append(c, ks, vs, at, lengths, n, dtype, **kw):
    """Appends the tokens [at[b], at[b] + n) of each sequence, those it has."""
    B, _, H, D = c.k.shape
    new = [max(0, min(n, len(x) - a)) for x, a in zip(ks, at)]

    def pack(xs):
        y = np.full((B, n, H, D), 7.0)
        for b, x in enumerate(xs):
            y[b, :new[b]] = x[at[b]:at[b] + new[b]]
        return dev(y, dtype)

    pamm.cache_append_fp8(c, pack(ks), pack(vs), lengths, new_len=lens(new) if min(new) < n else None, **kw)
    return [a + m for a, m in zip(at, new)]


def build(B, room, H, D, block, dtype, lengths, chunks, seed=0):
    rng = np.random.default_rng(seed)
    c = filled(B, room, H, D, block, dtype)
    ks, vs = (rounded(tokens(rng, lengths, H, D, dtype), dtype) for _ in "kv")
    at, n = [0] * B, lens([0] * B)
    for chunk in chunks:
        at = append(c, ks, vs, at, n, chunk, dtype)
        assert n.tolist() == at
    assert at == list(lengths)
    return c, ks, vs, n


@BOTH
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("D", [16, 48, 80, 128])
def test_append(dtype, block, D):
    """Lengths around a block, in one call, token by token and in odd chunks: the same cache."""
    say("append", dtype, block, D)
    lengths = [0, 1, block - 1, block, block + 1, 2 * block, 3 * block - 1]
    room, caches = 3 * block + 5, []
    for chunks in ([3 * block], [1] * (3 * block), [block // 2 - 1, 2, block, 7] + [19] * (block // 8)):
        c, ks, vs, n = build(7, room, 3, D, block, dtype, lengths, chunks)
        holds(c, "k", ks, dtype)
        holds(c, "v", vs, dtype)
        caches.append(c)
    for other in caches[1:]:
        assert all(np.array_equal(raw(a), raw(b)) for a, b in zip(caches[0][:2], other[:2]))
        assert all(torch.equal(a[:, :1], b[:, :1]) for a, b in zip(caches[0][2:4], other[2:4]))


@BOTH
@pytest.mark.parametrize("B,H,n", [(1, 1, 1), (64, 8, 1), (2, 32, 333), (1, 2, 5000)])
def test_append_sizes(dtype, B, H, n):
    say("append", dtype, B, H, n)
    c, ks, vs, _ = build(B, n + 3, H, 64, 32, dtype, [n] * B, [n])
    holds(c, "k", ks, dtype)
    holds(c, "v", vs, dtype)


@BOTH
def test_tokens_past_the_room_are_dropped(dtype):
    rng = np.random.default_rng(1)
    for room in (96, 100):
        c = filled(3, room, 2, 32, 32, dtype)
        ks, vs = (rounded(tokens(rng, [130] * 3, 2, 32, dtype), dtype) for _ in "kv")
        n = lens([0] * 3)
        pack = lambda xs: dev(np.stack(xs), dtype)
        pamm.cache_append_fp8(c, pack(ks)[:, :50], pack(vs)[:, :50], n)
        pamm.cache_append_fp8(c, pack(ks)[:, 50:], pack(vs)[:, 50:], n)
        assert n.tolist() == [room] * 3
        # the tail's first rows held older tokens, which holds() compares only up to the length
        holds(c, "k", [x[:room] for x in ks], dtype)
        before = [raw(t).copy() for t in c]
        pamm.cache_append_fp8(c, pack(ks), pack(vs), n)
        assert n.tolist() == [room] * 3 and all(np.array_equal(raw(t), b) for t, b in zip(c, before))
        for bad in (-5, room + 1000):  # lengths outside the room count as its ends
            c2 = filled(3, room, 2, 32, 32, dtype)
            m = lens([bad] * 3)
            pamm.cache_append_fp8(c2, pack(ks)[:, :40], pack(vs)[:, :40], m, new_len=lens([-1, 40, 99]))
            if bad < 0:
                assert m.tolist() == [0, 40, 40]
                holds(c2, "v", [vs[0][:0], vs[1][:40], vs[2][:40]], dtype)
            else:
                assert m.tolist() == [room] * 3 and all(marked(t) for t in (c2.k, c2.v, c2.k_tail, c2.v_tail))


def test_lengths_stay_without_advance():
    c, n = pamm.CacheFP8.empty(2, 64, 1, 16, block=32), lens([3, 40])
    x = torch.ones(2, 5, 1, 16, device="cuda", dtype=torch.bfloat16)
    pamm.cache_append_fp8(c, x, x, n, advance=False)
    assert n.tolist() == [3, 40] and (c.k_tail[0, 3:8] == 1).all() and (c.k_tail[1, 8:13] == 1).all()
    pamm.cache_append_fp8(c, x[:, :0], x[:, :0], n)
    assert n.tolist() == [3, 40]


@BOTH
def test_extreme_values(dtype):
    """Blocks of zeros, of the type's least and largest numbers, and with what is not finite."""
    say("append extremes", dtype)
    rng = np.random.default_rng(2)
    x = values(rng, (7 * 32, 2, 16), dtype)
    x[32:64] = 0
    x[64:96] *= 2.0 ** -130
    x[96:128] *= 2.0 ** 124
    x[130, 0, 3], x[140, 1, 5], x[150, 0, 9] = np.nan, np.inf, -np.inf
    x[160:192] = np.nan
    x[192:224, :, :] = 448 * 2.0 ** -4
    x[192:224, :, 1:] = 17 * 2.0 ** -4  # half way between 16 and 18 scales: to even, 16
    x = rounded([x], dtype)
    c, n = filled(1, 7 * 32, 2, 16, 32, dtype), lens([0])
    pamm.cache_append_fp8(c, dev(x[0][None], dtype), dev(x[0][None], dtype), n)
    holds(c, "k", x, dtype)
    holds(c, "v", x, dtype)
    q, s = host(c.k.float())[0], host(c.k_scale)[0]
    assert not q[32:64].any() and (s[1] == 2.0 ** -126).all() and np.isnan(q[160:192]).all()
    assert (q[192:224, :, 1:] == 16).all() and (q[192:224, :, 0] == 448).all()


@BOTH
def test_any_layout(dtype):
    """Caches and new tokens in any order of the outer dimensions."""
    rng = np.random.default_rng(3)
    B, room, H, D, block = 2, 96, 3, 32, 32
    ks, vs = (rounded(tokens(rng, [90, 90], H, D, dtype), dtype) for _ in "kv")
    want = filled(B, room, H, D, block, dtype)
    n = lens([0, 0])
    kd, vd = dev(np.stack(ks), dtype), dev(np.stack(vs), dtype)
    pamm.cache_append_fp8(want, kd, vd, n)
    q = torch.randn(B, 4, 6, D, device="cuda").to(DT[dtype])
    o, lse = pamm.attention_fp8(q, want, n, causal=True)
    for perm in ((0, 1, 2, 3), (1, 0, 2, 3), (2, 1, 0, 3)):
        back = [perm.index(i) for i in range(4)]

        def place(t):
            return torch.zeros([t.shape[i] for i in perm], dtype=t.dtype, device="cuda").permute(back)

        c = pamm.CacheFP8(*(place(t) for t in (want.k, want.v)),
                          *(torch.zeros(H, B, room // block, device="cuda").permute(1, 2, 0) for _ in range(2)),
                          *(place(t) for t in (want.k_tail, want.v_tail)))
        m = lens([0, 0])
        moved = [place(t).copy_(t) for t in (kd, vd)]
        pamm.cache_append_fp8(c, *moved, m)
        for got, ref in zip(c[:2], want[:2]):
            assert torch.equal(got[:, :64].float(), ref[:, :64].float())
        assert torch.equal(c.k_scale[:, :2], want.k_scale[:, :2]) and torch.equal(c.v_tail[:, :26], want.v_tail[:, :26])
        o2, lse2 = pamm.attention_fp8(place(q).copy_(q), c, m, causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@BOTH
def test_the_last_tokens_can_be_taken_back(dtype):
    """Lengths lowered as far as the end of the last whole block, and other tokens appended behind them."""
    rng = np.random.default_rng(3)
    first, second = (rounded(tokens(rng, [80, 75], 2, 32, dtype), dtype) for _ in range(2))
    c, n = filled(2, 160, 2, 32, 64, dtype), lens([0, 0])
    kv = [dev(np.stack([x[:75] for x in xs]), dtype) for xs in (first, second)]
    pamm.cache_append_fp8(c, kv[0], kv[1], n)
    n.copy_(lens([70, 64]))
    pamm.cache_append_fp8(c, kv[1][:, :70], kv[0][:, :70], n)
    assert n.tolist() == [140, 134]
    for name, a, b in (("k", first, second), ("v", second, first)):
        want = [np.concatenate([a[0][:70], b[0][:70]]), np.concatenate([a[1][:64], b[1][:70]])]
        holds(c, name, want, dtype)


# ------------------------------------------------------------------ attention

def meant(c, lengths, room):
    """What the cache's bytes stand for, [B, room, H, D] each."""
    res = []
    block = c.k_tail.shape[1]
    for eight, scale, tail in ((c.k, c.k_scale, c.k_tail), (c.v, c.v_scale, c.v_tail)):
        x = np.zeros((eight.shape[0], room) + tuple(eight.shape[2:]))
        e, s, t = host(eight.float()), host(scale), host(tail.float())
        for b, L in enumerate(lengths):
            whole = L // block * block
            x[b, :whole] = e[b, :whole] * np.repeat(s[b, :whole // block], block, 0)[..., None]
            x[b, whole:L] = t[b, :L - whole]
        res.append(x)
    return res


def check(B, Sq, lengths, H, Hkv, D, block, dtype, *, room=None, seed=0, spoil=None, sliced=False, **kw):
    say("attention_fp8", B, Sq, lengths, H, Hkv, D, block, dtype, kw)
    room = room or max(max(lengths), 1)
    c, _, _, n = build(B, room, Hkv, D, block, dtype, lengths, [max(lengths)] if max(lengths) else [], seed=seed)
    if spoil:
        spoil(c)
    k, v = meant(c, lengths, room)
    rng = np.random.default_rng(seed + 1)
    q = values(rng, (B, Sq, H, D), dtype)
    rk = dict(kw, kv_len=lengths)
    ref = bo.attention(q, k, v, dtype=dtype, **rk)
    gk = dict(kw, q_len=lens(kw.get("q_len")))
    seen = c._replace(k=c.k[:, :max(lengths)], v=c.v[:, :max(lengths)]) if sliced else c
    o, lse = pamm.attention_fp8(dev(q, dtype), seen, n, **gk)
    # over attention's bounds: the values' scale is one more product of each probability
    more = 4 * bo.U * np.abs(np.where(np.isfinite(v), v, 0.0)).max(initial=0.0)
    close("o", o, ref["o"], ref["o_tol"] + more)
    close("lse", lse, ref["lse"], ref["lse_tol"])
    again, _ = pamm.attention_fp8(dev(q, dtype), seen, n, **gk)
    assert torch.equal(o, again) or not torch.isfinite(o).all()
    return o, lse


@BOTH
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
def test_head_dims(dtype, D):
    check(2, 1, [70, 33], 4, 2, D, 32, dtype, causal=True)
    check(2, 40, [140, 65], 4, 2, D, 32, dtype, causal=True)


@BOTH
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("Sq", [1, 3, 40, 130])
def test_lengths(dtype, block, Sq):
    """0, 1, and around whole blocks; fewer keys than queries among them."""
    check(8, Sq, [0, 1, block - 1, block, block + 1, 2 * block - 1, 2 * block, 3 * block + 17], 6, 2, 64, block, dtype,
          causal=True, room=4 * block)


@BOTH
@pytest.mark.parametrize("H,Hkv", [(1, 1), (12, 12), (32, 1), (33, 1), (80, 2), (8, 4)])
def test_heads(dtype, H, Hkv):
    check(2, 1, [300, 77], H, Hkv, 32, 64, dtype, causal=True)


@BOTH
@pytest.mark.parametrize("window", [1, 5, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("Sq", [1, 2, 70])
def test_windows(dtype, window, Sq):
    check(3, Sq, [257, 100, 640], 4, 2, 32, 32, dtype, causal=True, window=window)


@BOTH
@pytest.mark.parametrize("Sq", [1, 5, 70])
def test_without_causal_mask(dtype, Sq):
    check(2, Sq, [129, 300], 4, 2, 64, 64, dtype)
    check(2, Sq, [129, 300], 4, 4, 64, 64, dtype, scale=-0.3)


@BOTH
def test_query_lengths(dtype):
    check(4, 37, [100, 100, 64, 0], 4, 2, 32, 32, dtype, causal=True, q_len=[37, 5, 0, 37])


@BOTH
@pytest.mark.parametrize("B,Sq,L", [(1, 1, 9000), (3, 1, 4000), (1, 9, 5000), (1, 200, 3000)])
def test_split_keys(dtype, B, Sq, L):
    """Long caches, which are cut over the device and joined."""
    check(B, Sq, [max(Sq, L - 777 * b) for b in range(B)], 4, 1, 64, 128, dtype, causal=True)


@BOTH
def test_sliced_cache(dtype):
    check(2, 1, [70, 65], 4, 2, 32, 32, dtype, room=500, causal=True, sliced=True)
    check(2, 40, [96, 90], 4, 2, 32, 32, dtype, room=500, causal=True, sliced=True)


def test_no_lengths():
    """All rows are valid; the last, partial block is the tail's."""
    c, _, _, n = build(2, 100, 2, 32, 32, "f32", [100, 100], [100])
    q = torch.randn(2, 3, 4, 32, device="cuda")
    a, b = pamm.attention_fp8(q, c, n, causal=True), pamm.attention_fp8(q, c, None, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@BOTH
@pytest.mark.parametrize("Sq", [1, 4, 70])
@pytest.mark.parametrize("place", ["eight", "tail"])
def test_hidden_values_do_not_come_through(dtype, Sq, place):
    """A NaN (in the tail also an infinity) in keys and values that a window or the causal mask hides from some
    queries: rows that do not see it are as the definition says, those that do see it are not finite."""
    L = 150  # 128 in 8 bits
    at = 100 if place == "eight" else 140

    def spoil(c):
        if place == "eight":
            c.k[0, at, 0, 3], c.v[0, at, 0, 5] = float("nan"), float("nan")
        else:
            c.k_tail[0, at - 128, 0, 3], c.v_tail[0, at - 128, 0, 5] = float("nan"), float("inf")

    window = 8 if Sq == 1 or place == "tail" else 30
    sees = np.array([L - Sq + i >= at > L - Sq + i - window for i in range(Sq)])
    say("hidden", dtype, Sq, place, int(sees.sum()), "see it")
    c, _, _, n = build(1, L, 1, 32, 32, dtype, [L], [L])
    spoil(c)
    # the definition with 0 in its place, for the rows that do not see it
    k, v = (np.where(np.isfinite(x), x, 0.0) for x in meant(c, [L], L))
    q = values(np.random.default_rng(1), (1, Sq, 2, 32), dtype)
    ref = bo.attention(q, k, v, dtype=dtype, causal=True, window=window, kv_len=[L])
    o, lse = pamm.attention_fp8(dev(q, dtype), c, n, causal=True, window=window)
    more = 4 * bo.U * np.abs(v).max()
    close("o", host(o)[:, ~sees], ref["o"][:, ~sees], ref["o_tol"][:, ~sees] + more)
    close("lse", host(lse)[..., ~sees], ref["lse"][..., ~sees], ref["lse_tol"][..., ~sees])
    assert torch.isnan(o[:, torch.from_numpy(sees).cuda()]).all()  # a NaN in the key makes the score NaN


@BOTH
@pytest.mark.parametrize("Sq", [1, 40])
def test_what_lies_behind_the_length_is_never_seen(dtype, Sq):
    """NaN bytes and scales behind the last whole block, and in the tail behind the last token."""
    def spoil(c):
        c.k.view(torch.uint8)[:, 64:] = 0x7F
        c.v.view(torch.uint8)[:, 64:] = 0x7F
        c.k_scale[:, 2:] = float("nan")
        c.v_scale[:, 2:] = float("nan")
        c.k_tail[:, 9:] = float("nan")
        c.v_tail[:, 9:] = float("inf")

    o, _ = check(2, Sq, [73, 73], 4, 2, 32, 32, dtype, room=160, spoil=spoil, causal=True)
    assert torch.isfinite(o).all()


@BOTH
@pytest.mark.parametrize("Sq,H,Hkv", [(1, 4, 2), (1, 20, 1), (40, 2, 1), (200, 2, 1)])
@pytest.mark.parametrize("window", [0, 20])
def test_scales_far_apart(dtype, Sq, H, Hkv, window):
    """Values of neighbouring blocks up to 2^150 apart, blocks of zeros among them: the window leaves some queries
    nothing but small ones, whose results have to be as exact as the others'."""
    block, n = 32, 24
    rng = np.random.default_rng(5)
    powers = rng.permutation([0, -3, -9, -11, -14, -24, -26, -45, -60, -90, 20, 50, 60, 5, 0, -1, -100, 30, -50, 1, 0, 0, 2, -7])
    L = block * n + 7
    ks = [values(rng, (L, Hkv, 32), dtype)]
    vs = [values(rng, (L, Hkv, 32), dtype)]
    for i, p in enumerate(powers):
        vs[0][i * block:(i + 1) * block] *= 2.0 ** p
    vs[0][3 * block:4 * block] = 0
    ks, vs = rounded(ks, dtype), rounded(vs, dtype)
    c, at = filled(1, L, Hkv, 32, block, dtype), lens([0])
    pamm.cache_append_fp8(c, dev(ks[0][None], dtype), dev(vs[0][None], dtype), at)
    k, v = meant(c, [L], L)
    for end in (L, L - 7, 5 * block, 11 * block + 3):
        say("scales", dtype, Sq, H, window, end)
        n_q = min(Sq, end)
        q = values(np.random.default_rng(6), (1, n_q, H, 32), dtype)
        whole = end // block * block
        kk, vv = k.copy(), v.copy()
        if end < L:  # the tail is that of the whole cache: put the block's tokens there
            for x, t in ((kk, c.k_tail), (vv, c.v_tail)):
                x[0, whole:end] = host(t.float())[0, :end - whole]
        ref = bo.attention(q, kk, vv, dtype=dtype, causal=True, window=window, kv_len=[end])
        o, lse = pamm.attention_fp8(dev(q, dtype), c, lens([end]), causal=True, window=window)
        # one more product for each probability: 4 u of a row's sum of P |v|, which the bound's P part holds 2^-8
        # or E >= 16 u of
        close("o", o, ref["o"], 1.5 * ref["o_tol"])
        close("lse", lse, ref["lse"], ref["lse_tol"])


@BOTH
@pytest.mark.parametrize("Sq", [1, 8, 12, 130])
@pytest.mark.parametrize("scale", [0.0, 1e-12, None])
def test_blocks_of_zeros(dtype, Sq, scale):
    """Their scale is the least one, whose product with a small factor of the scores leaves fp32's range: masked
    scores stay masked, the others 0."""
    say("zeros", dtype, Sq, scale)
    L = 140
    c, _, _, n = build(1, L, 1, 32, 64, dtype, [L], [L])
    c.k[:, 64:128] = 0
    c.k_scale[:, 1] = 2.0 ** -126
    k, v = meant(c, [L], L)
    q = values(np.random.default_rng(1), (1, Sq, 2, 32), dtype)
    kw = dict(causal=True, window=30)
    if scale is not None:
        kw["scale"] = scale
    ref = bo.attention(q, k, v, dtype=dtype, kv_len=[L], **kw)
    o, lse = pamm.attention_fp8(dev(q, dtype), c, n, **kw)
    close("o", o, ref["o"], ref["o_tol"] + 4 * bo.U * np.abs(v).max())
    close("lse", lse, ref["lse"], ref["lse_tol"])


def test_far_rows():
    """Byte offsets past 2^32: two sequences of 8-bit rows more than that apart, and a long one."""
    big = torch.empty((1 << 32) + (1 << 20), dtype=torch.uint8, device="cuda")
    small = build(2, 320, 1, 64, 64, "bf16", [300, 311], [311])[0]
    n, q = lens([300, 311]), torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
    want = pamm.attention_fp8(q, small, n)
    k = big.view(torch.float8_e4m3fn).as_strided((2, 320, 1, 64), (1 << 32, 64, 64, 1), 0)
    v = big.view(torch.float8_e4m3fn).as_strided((2, 320, 1, 64), (1 << 31, 3 * (1 << 20), 64, 1), 1 << 19)
    k.view(torch.uint8).copy_(small.k.view(torch.uint8))
    v.view(torch.uint8).copy_(small.v.view(torch.uint8))
    got = pamm.attention_fp8(q, small._replace(k=k, v=v), n)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del big, k, v
    # one sequence of 2^25 + 100 tokens of 128 bytes: the last keys lie past 2^32
    L, room = (1 << 25) + 100, (1 << 25) + 128
    long = pamm.CacheFP8.empty(1, room, 1, 128, block=128)
    part = torch.randn(1, 228, 1, 128, device="cuda").bfloat16()
    at = lens([L - 228])
    pamm.cache_append_fp8(long, part, part, at)
    assert at.tolist() == [L]
    q = torch.randn(1, 1, 2, 128, device="cuda").bfloat16()
    got = pamm.attention_fp8(q, long, at, causal=True, window=200)
    near = pamm.CacheFP8.empty(1, 384, 1, 128, block=128)
    m = lens([0])
    pamm.cache_append_fp8(near, torch.cat([part[:, :128], part], 1), torch.cat([part[:, :128], part], 1), m)
    want = pamm.attention_fp8(q, near, m, causal=True, window=200)
    # the same keys, cut into parts elsewhere: 2^-8 of the value for the rounding, as much for P's
    assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -6 * part.abs().max()
    assert (got[1] - want[1]).abs().max() < 1e-4


def test_workspace_stream_and_outputs():
    c, _, _, n = build(2, 4096, 2, 64, 64, "bf16", [4000, 3001], [4000])
    q = torch.randn(2, 1, 8, 64, device="cuda").bfloat16()
    need = pamm.attention_fp8_workspace_size(q, c, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o, lse = pamm.attention_fp8(q, c, n, causal=True)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    pamm.attention_fp8(q, c, n, causal=True, o=o2, lse=lse2, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises(ValueError, match="workspace"):
        pamm.attention_fp8(q, c, n, workspace=ws[:64])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pamm.attention_fp8(q, c, n, causal=True, stream=side)
    side.synchronize()
    assert torch.equal(got[0], o)
    x = torch.randn(2, 1, 2, 64, device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    pamm.cache_append_fp8(c, x, x, n, stream=side)
    side.synchronize()
    assert n.tolist() == [4001, 3002] and torch.equal(c.k_tail[0, 4000 % 64], x[0, 0])


def test_empty_calls():
    c = pamm.CacheFP8.empty(2, 0, 1, 16)
    q = torch.randn(2, 3, 2, 16, device="cuda").bfloat16()
    o, lse = pamm.attention_fp8(q, c, lens([0, 0]), causal=True)
    assert not o.any() and torch.isneginf(lse).all()
    o, lse = pamm.attention_fp8(q[:0], pamm.CacheFP8.empty(0, 64, 1, 16), None)
    assert o.shape == (0, 3, 2, 16)
    o, lse = pamm.attention_fp8(q[:, :0], pamm.CacheFP8.empty(2, 64, 1, 16), lens([0, 0]))
    assert o.shape == (2, 0, 2, 16)
