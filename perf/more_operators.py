"""Operators between a PAMM projection and its attention, as cases that can be
timed and checked: rotary positions, norms of queries and keys with the
rotation in the same pass (forward and gradients), and a cache of keys and
values in 8 bits with a scale for each block of tokens and head: appending to
it and attention over it.

With `own` false `run` computes the plain form: elementary torch operations in
32 bits (angles in 64), rounded once at the end.  With `own` true it calls this
package.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def _rot(name, op, B, S, H, Hkv, D, dtype, R=None, inter=False, far=0, pos="none", inverse=False, stretch=1.0):
    """far: the first position; pos: how positions are given (none, offset, each)."""
    c = {"op": op, "B": B, "S": S, "H": H, "Hkv": Hkv, "D": D, "dtype": dtype, "R": R or D, "inter": inter, "far": far,
         "pos": pos, "inverse": inverse, "stretch": stretch}
    return dict(c, name=name) if name else c


def _cache(name, op, B, n, room, H, Hkv, D, T, dtype, ragged, window=0):
    c = {"op": op, "B": B, "n": n, "room": room, "H": H, "Hkv": Hkv, "D": D, "T": T, "dtype": dtype, "ragged": ragged,
         "window": window}
    return dict(c, name=name) if name else c


def listed():
    return [
        # training behind the 4096-wide projection, 2048-token sequences: queries and keys of the packed output
        _rot("rotary_b4_s2048_d128", "rotary", 4, 2048, 32, 32, 128, "bf16"),
        # the gradient of a long sequence's rotation, shared key/value heads, interleaved pairs, a stretched context
        _rot("rotary_grad_s8192_d64", "rotary", 1, 8192, 32, 8, 64, "bf16", inter=True, far=100000, pos="offset",
             inverse=True, stretch=4.0),
        # odd sizes in 32 bits: half of each head rotated, pairs that no vector holds, a position for each token
        _rot("rotary_partial_f32", "rotary", 3, 333, 6, 2, 40, "f32", R=20, far=1000000, pos="each", stretch=8.0),
        # serving, the smallest call: one sequence's new token
        _rot("qknorm_token_b1", "qknorm", 1, 1, 12, 12, 64, "bf16", far=129, pos="offset"),
        # one training step of the 768-wide model: 12 heads of 64, 1024 tokens
        _rot("qknorm_step_s1024_d64", "qknorm_step", 8, 1024, 12, 12, 64, "bf16"),
        # one training step with shared key/value heads, 4096-wide, part of each head rotated
        _rot("qknorm_step_gqa_d128", "qknorm_step", 4, 2048, 32, 8, 128, "bf16", R=64, inter=True, pos="each", far=17),
        # serving, a full batch: one new token each; some of them complete a block
        _cache("append_token_b64", "append", 64, 1, 2048, 32, 8, 128, 64, "bf16", True),
        # serving: prompts of up to 2048 tokens into an empty cache
        _cache("append_prompt_b4_s2048", "append", 4, 2048, 2048, 32, 32, 128, 32, "bf16", True),
        # serving, the smallest call: one sequence, one new token, a short cache
        _cache("attn8_token_b1_s130", "attn8", 1, 1, 130, 12, 12, 64, 64, "bf16", False),
        # serving, a full batch: one new token each over long caches of different lengths
        _cache("attn8_token_b64_s8192", "attn8", 64, 1, 8192, 32, 8, 128, 64, "bf16", True),
        # serving: a chunk of 512 new tokens against the cache before it
        _cache("attn8_chunk_512_over_8192", "attn8", 2, 512, 8192, 32, 8, 128, 32, "bf16", False),
        # odd sizes in 32 bits, sequences of different lengths, sliding window
        _cache("attn8_f32_window", "attn8", 3, 37, 1001, 6, 2, 48, 32, "f32", True, 100),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "qknorm", "qknorm_step", "qknorm_step", "append", "append", "attn8", "attn8",
                     "attn8"])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 4])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("rotary", "qknorm", "qknorm_step"):
        D = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
        R = rng.choice([D, D, D, D // 2, D // 4 * 2 - 2])
        S = _log_int(rng, 1, 4000)
        B = _log_int(rng, 1, max(1, min(8, 8192 // S)))
        return _rot(None, op, B, S, H, Hkv, D, dtype, R, rng.random() < 0.4, rng.choice([0, _log_int(rng, 1, 2000000)]),
                    rng.choice(["none", "offset", "each"]), op == "rotary" and rng.random() < 0.5,
                    rng.choice([1.0, 1.0, rng.uniform(1.5, 16.0)]))
    D, T = rng.choice([32, 48, 64, 64, 80, 96, 112, 128, 128]), rng.choice([32, 64, 128])
    ragged = rng.random() < 0.6
    if op == "append":
        if rng.random() < 0.5:
            return _cache(None, op, _log_int(rng, 1, 64), 1, _log_int(rng, 130, 2000), H, Hkv, D, T, dtype, ragged)
        n = _log_int(rng, 2, 2000)
        return _cache(None, op, _log_int(rng, 1, 4), n, n + _log_int(rng, 1, 2000), H, Hkv, D, T, dtype, ragged)
    if rng.random() < 0.6:
        return _cache(None, op, _log_int(rng, 1, 64), 1, _log_int(rng, 1, 8000), H, Hkv, D, T, dtype, ragged)
    B, n = _log_int(rng, 1, 4), _log_int(rng, 2, 512 if dtype == "bf16" else 100)
    room = n + _log_int(rng, 1, 7000 if dtype == "bf16" else 2000)
    while B > 1 and B * n * room * H * D > 2 * 512 * 8192 * 32 * 128:
        B //= 2
    return _cache(None, op, B, n, room, H, Hkv, D, T, dtype, ragged, _log_int(rng, 8, room) if rng.random() < 0.3 else 0)


def _lengths(c, seed):
    """attn8: the valid keys of each sequence, the new tokens among them.
    append: (tokens before, new tokens).  A chunk of more than one token starts
    at a whole block here, so that a pass can be repeated on its own result."""
    B, n, room, T = c["B"], c["n"], c["room"], c["T"]
    rng = random.Random(seed)
    if c["op"] == "attn8":
        lens = [max(n, room - (b * room) // (B + 1)) if c["ragged"] else room for b in range(B)]
        rng.shuffle(lens)
        return lens
    if n == 1:
        start = [rng.randrange(room) if c["ragged"] else room - 1 for _ in range(B)]
        return start, [1] * B
    start = [rng.randrange((room - n) // T + 1) * T if c["ragged"] else 0 for _ in range(B)]
    return start, [max(1, n - (b * n) // (B + 1)) if c["ragged"] else n for b in range(B)]


# ----------------------------------------------------------------- the inputs

def _blocks(x, T):
    """[B, H, S, D] with S a multiple of T -> 8-bit values and scales [B, H, S / T]."""
    B, H, S, D = x.shape
    y = x.float().reshape(B, H, S // T, T * D)
    scale = (y.abs().amax(3) / 448.0).clamp(min=2.0 ** -126)
    q = (y / scale[..., None]).clamp(-448, 448).to(F8)
    return q.reshape(B, H, S, D), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 5)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    dt, B, H, Hkv, D = DT[c["dtype"]], c["B"], c["H"], c["Hkv"], c["D"]
    s = {"case": c}
    if c["op"] in ("rotary", "qknorm", "qknorm_step"):
        S, R = c["S"], c["R"]
        # what a program keeps: radians a position for each pair, in 64 bits; a stretched context slows the low ones
        f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        s["inv_freq"] = torch.where(f * 8192 < 2 * math.pi, f / c["stretch"], f)
        s["magnitude"] = 1.0 + 0.1 * math.log(c["stretch"])
        s["positions"] = s["offset"] = None
        if c["pos"] == "offset":
            s["offset"] = (c["far"] + torch.randint(0, 1000, (B,), generator=g, device="cuda")).int()
        elif c["pos"] == "each":  # documents packed into one row: positions start again somewhere
            cut = torch.randint(0, S, (B, 1), generator=g, device="cuda")
            i = torch.arange(S, device="cuda")[None]
            s["positions"] = torch.where(i < cut, i, i - cut + c["far"])
        qkv = randn(B, S, H + 2 * Hkv, D, dtype=dt)  # the packed output of the projection
        qkv[..., :: max(1, D // 3)] *= 4  # a few large channels
        s["qk"] = qkv[:, :, :H + Hkv]
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        if c["op"] != "rotary":
            s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
            s["eps"] = 1e-6
        if c["op"] == "qknorm_step":
            s["dq"], s["dk"] = randn(B, S, H, D, dtype=dt), randn(B, S, Hkv, D, dtype=dt)
        return s
    n, T = c["n"], c["T"]
    room = (c["room"] + T - 1) // T * T + (T if c["op"] == "append" else 0)
    # heads of different sizes, a few large channels, as keys have
    size = torch.rand(Hkv, 1, 1, generator=g, device="cuda") + 0.5
    for name in ("k", "v"):
        x = randn(B, Hkv, room, D, dtype=torch.bfloat16) * size.bfloat16()
        x[..., :: max(1, D // 3)] *= 4 if name == "k" else 1
        q, scale = _blocks(x, T)
        del x
        s[name + "8"] = q.transpose(1, 2)                    # [B, room, Hkv, D]
        s[name + "_scale"] = scale.transpose(1, 2)           # [B, room / T, Hkv]
        s[name + "_tail"] = randn(B, Hkv, T, D, dtype=dt).transpose(1, 2)  # [B, T, Hkv, D]
    if c["op"] == "attn8":
        s["q"] = randn(B, n, H, D, dtype=dt)
        s["kv_len"] = torch.tensor(_lengths(c, seed), dtype=torch.int32, device="cuda")
        return s
    start, new = _lengths(c, seed)
    s["lengths"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["new_len"] = torch.tensor(new, dtype=torch.int32, device="cuda") if c["ragged"] and n > 1 else None
    qkv = randn(B, n, H + 2 * Hkv, D, dtype=dt)
    s["k"], s["v"] = qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    return s


# ---------------------------------------------------------------- plain forms

def _plain_angles(c, s):
    pos = torch.arange(c["S"], device="cuda")[None].expand(c["B"], -1) if s["positions"] is None else s["positions"]
    if s["offset"] is not None:
        pos = pos + s["offset"][:, None]
    t = pos[..., None].double() * s["inv_freq"]
    m = s["magnitude"]
    return (t.cos() * m).float()[:, :, None], (t.sin() * m).float()[:, :, None]


def _plain_rotate(c, x, cos, sin):
    R = c["R"]
    if c["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
    a, b = a * cos - b * sin, a * sin + b * cos
    if c["inter"]:
        y = torch.stack([a, b], -1).flatten(-2)
    else:
        y = torch.cat([a, b], -1)
    return torch.cat([y, x[..., R:]], -1) if R < c["D"] else y


def _plain_rotary(c, s):
    dt = DT[c["dtype"]]
    cos, sin = _plain_angles(c, s)
    if c["op"] == "rotary":
        return {"out": _plain_rotate(c, s["qk"].float(), cos, -sin if c["inverse"] else sin).to(dt)}
    res = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n].float()
        rstd = torch.rsqrt(x.square().mean(3, keepdim=True) + s["eps"])
        xhat = x * rstd
        res[n] = _plain_rotate(c, xhat * w, cos, sin).to(dt)
        if c["op"] == "qknorm_step":
            gn = _plain_rotate(c, s["d" + n].float(), cos, -sin)
            u = gn * w
            res["d" + n] = (rstd * (u - xhat * (u * xhat).mean(3, keepdim=True))).to(dt)
            res["dw" + n] = (gn * xhat).sum((0, 1, 2))
    return res


def _plain_append(c, s):
    B, n, T, H, D = c["B"], c["n"], c["T"], c["Hkv"], c["D"]
    start = s["lengths"].long()
    new = s["new_len"].long() if s["new_len"] is not None else torch.full_like(start, n)
    into = start % T                      # tokens that wait in the tail
    nb = (n + T - 2) // T + 1             # blocks that n tokens can touch
    at = torch.arange(nb * T, device="cuda")[None]
    src = at - into[:, None]              # new token of each place in the touched blocks
    b = torch.arange(B, device="cuda")[:, None]
    end = into + new
    res = {}
    for name in ("k", "v"):
        x, tail = s[name], s[name + "_tail"]
        old = (src < 0)[..., None, None]
        rows = torch.where(old, tail[b, at % T], x[b, src.clamp(0, n - 1)])
        live = (at < end[:, None])[..., None, None]
        y = torch.where(live, rows, 0).float().reshape(B, nb, T, H, D)
        scale = (y.abs().amax((2, 4)) / 448.0).clamp(min=2.0 ** -126)
        q = (y / scale[:, :, None, :, None]).clamp(-448, 448).to(F8)
        whole = (torch.arange(nb, device="cuda")[None] + 1) * T <= end[:, None]
        store, scales = s[name + "8"], s[name + "_scale"]
        blocks = store.view(torch.uint8).transpose(1, 2).reshape(B, H, -1, T, D)  # a view: heads lie first
        to = (start // T)[:, None] + torch.arange(nb, device="cuda")[None]
        byte = q.view(torch.uint8).permute(0, 1, 3, 2, 4)
        blocks[b, :, to] = torch.where(whole[..., None, None, None], byte, blocks[b, :, to])
        scales[b, to] = torch.where(whole[..., None], scale, scales[b, to])
        # the tokens behind the last whole block
        first = end // T * T
        slot = torch.arange(T, device="cuda")[None]
        src2 = first[:, None] + slot - into[:, None]
        keep = (first[:, None] + slot >= end[:, None]) | (src2 < 0)
        s[name + "_tail"].copy_(torch.where(keep[..., None, None], tail, x[b, src2.clamp(0, n - 1)]))
        res.update({name + "8": store, name + "_scale": scales, name + "_tail": s[name + "_tail"]})
    return res


def _plain_attn8(c, s):
    B, n, H, Hkv, D, T, dt = c["B"], c["n"], c["H"], c["Hkv"], c["D"], c["T"], DT[c["dtype"]]
    G, room = H // Hkv, s["k8"].shape[1]
    i = torch.arange(n, device="cuda")[None, :, None]
    j = torch.arange(room, device="cuda")[None, None]
    kl = s["kv_len"][:, None, None]
    mask = (j < kl) & (j <= i + (kl - n))
    if c["window"]:
        mask = mask & (j > i + (kl - n) - c["window"])
    whole = (s["kv_len"] // T * T)[:, None]
    place = torch.arange(room, device="cuda")[None]

    def values(name):
        x = s[name + "8"].transpose(1, 2).float().reshape(B, Hkv, room // T, T, D)
        x = (x * s[name + "_scale"].transpose(1, 2)[..., None, None]).reshape(B, Hkv, room, D)
        tail = s[name + "_tail"].transpose(1, 2).float()
        return torch.where((place >= whole)[:, None, :, None], tail.repeat(1, 1, room // T, 1), x)

    q = s["q"].float().transpose(1, 2).reshape(B, Hkv, G * n, D)
    sc = torch.matmul(q, values("k").transpose(2, 3)).mul_(D ** -0.5)
    sc.masked_fill_(~mask.repeat(1, G, 1)[:, None], -math.inf)
    top = sc.amax(3, keepdim=True)
    p = sc.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(3, keepdim=True)
    lse = (top + total.log()).reshape(B, H, n)
    o = torch.matmul(p.div_(total.clamp(min=1e-37)), values("v"))
    return {"o": o.reshape(B, H, n, D).transpose(1, 2).to(dt), "lse": lse}


# --------------------------------------------------------------------- a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return (_plain_append if c["op"] == "append" else _plain_attn8 if c["op"] == "attn8" else _plain_rotary)(c, s)
    import activation_compression_pamm_amd as pamm
    if c["op"] in ("append", "attn8"):
        cache = pamm.CacheFP8(s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"])
        if c["op"] == "attn8":
            o, lse = pamm.attention_fp8(s["q"], cache, s["kv_len"], causal=True, window=c["window"])
            return {"o": o, "lse": lse}
        pamm.cache_append_fp8(cache, s["k"], s["v"], s["lengths"], new_len=s["new_len"], advance=False)
        return {n: s[n] for n in ("k8", "k_scale", "k_tail", "v8", "v_scale", "v_tail")}
    kw = {"positions": s["positions"], "offset": s["offset"], "interleaved": c["inter"], "magnitude": s["magnitude"]}
    if c["op"] == "rotary":
        return {"out": pamm.rotary(s["qk"], s["inv_freq"], inverse=c["inverse"], **kw)}
    kw["eps"] = s["eps"]
    q, k = pamm.qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], **kw)
    if c["op"] == "qknorm":
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = pamm.qk_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"],
                                                    **kw)
    return {"q": q, "dq": dq, "dwq": dwq, "k": k, "dk": dk, "dwk": dwk}


# ------------------------------------------------------------------- the work

def work(case):
    c = case
    e, D, Hkv = 2 if c["dtype"] == "bf16" else 4, c["D"], c["Hkv"]
    if c["op"] in ("rotary", "qknorm", "qknorm_step"):
        tokens = c["B"] * c["S"]
        nd = tokens * (c["H"] + Hkv) * D
        where = {"none": 0, "offset": 4 * c["B"], "each": 8 * tokens}[c["pos"]]
        # x in, y out; the step also reads the output's gradient and writes the input's
        passes, flops = {"rotary": (2, 3), "qknorm": (2, 7), "qknorm_step": (4, 22)}[c["op"]]
        return {"bytes": passes * nd * e + where, "flops": flops * nd}
    T, n = c["T"], c["n"]
    if c["op"] == "attn8":
        lens = _lengths(c, 0)
        rows, total, pairs = 0, 0, 0
        for L in lens:  # the keys that some query sees
            low = max(0, L - n - c["window"] + 1) if c["window"] else 0
            whole = L // T * T
            total += 2 * Hkv * ((whole - min(low, whole)) * D + (L - max(whole, low)) * D * e)
            total += 2 * Hkv * 4 * (whole // T - min(low, whole) // T)
            pairs += sum(min(c["window"] or L, L - n + i + 1) for i in range(n))
        rows = c["B"] * n * c["H"]
        return {"bytes": total + rows * (2 * D * e + 4) + 4 * c["B"], "flops": 4 * D * c["H"] * pairs}
    start, new = _lengths(c, 0)
    total = flops = 0
    for a, m in zip(start, new):
        whole = (a + m) // T * T                       # tokens in whole blocks afterwards
        done = max(0, whole - a // T * T)              # those that this call turns into 8 bits
        waiting = a - a // T * T if done else 0        # of which the tail held
        total += 2 * Hkv * (D * e * (m + waiting) + D * done + 4 * (done // T) + D * e * (a + m - max(whole, a)))
        flops += 2 * Hkv * D * 3 * done
    return {"bytes": total + 8 * c["B"], "flops": flops}


# ------------------------------------------------------- the definition, 64 bits

def _exact_rotate(c, s, x, sign=1.0):
    """Each pair as a complex number times m exp(i angle)."""
    B, S = c["B"], c["S"]
    pos = torch.zeros(B, S, dtype=torch.float64, device="cuda")
    pos += torch.arange(S, device="cuda") if s["positions"] is None else s["positions"]
    if s["offset"] is not None:
        pos += s["offset"].double()[:, None]
    angle = sign * pos[:, :, None, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(angle, s["magnitude"]), angle)
    R, out = c["R"], x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if c["inter"] else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rotary(c, s):
    if c["op"] == "rotary":
        return {"out": _exact_rotate(c, s, s["qk"].double(), -1.0 if c["inverse"] else 1.0)}
    res = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        norm = torch.linalg.vector_norm(x, dim=3, keepdim=True)
        inv = 1 / torch.sqrt(norm * norm / c["D"] + s["eps"])
        res[n] = _exact_rotate(c, s, x * inv * w)
        if c["op"] == "qknorm_step":
            x.requires_grad_(True)
            w.requires_grad_(True)
            y = x * w / torch.sqrt(torch.einsum("bshd,bshd->bsh", x, x)[..., None] / c["D"] + s["eps"])
            gx, gw = torch.autograd.grad(y, (x, w), _exact_rotate(c, s, s["d" + n].double(), -1.0))
            res["d" + n], res["dw" + n] = gx, gw
    return res


def _e4m3(v):
    """The nearest value with 3 fraction bits, exponents from -6, largest 448; ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return (torch.round(v / unit) * unit).clamp(-448, 448)


def _exact_append(c, s):
    B, T = c["B"], c["T"]
    res = {}
    start = s["lengths"].tolist()
    new = s["new_len"].tolist() if s["new_len"] is not None else [c["n"]] * B
    for name in ("k", "v"):
        values, scales, tail = s[name + "8"].double(), s[name + "_scale"].double(), s[name + "_tail"].double()
        for b in range(B):
            wait = start[b] % T
            rows = torch.cat([tail[b, :wait], s[name][b, :new[b]].double()])
            first = start[b] // T
            while rows.shape[0] >= T:
                scale = torch.linalg.vector_norm(rows[:T], math.inf, dim=(0, 2)).clamp(min=448 * 2.0 ** -126) / 448
                values[b, first * T:(first + 1) * T] = _e4m3(rows[:T] / scale[None, :, None])
                scales[b, first] = scale
                rows, first = rows[T:], first + 1
            tail[b, :rows.shape[0]] = rows
        res.update({name + "8": values, name + "_scale": scales, name + "_tail": tail})
    return res


def _exact_attn8(c, s):
    """One (sequence, head) after another, its valid keys only."""
    B, n, H, Hkv, D, T = (c[x] for x in ("B", "n", "H", "Hkv", "D", "T"))
    if B * H > 3000:
        return None
    f64 = {"dtype": torch.float64, "device": "cuda"}
    o, lse = torch.zeros(B, n, H, D, **f64), torch.zeros(B, H, n, **f64)
    for b, L in enumerate(s["kv_len"].tolist()):
        whole = L // T * T
        last = torch.arange(n, device="cuda")[:, None] + L - n
        key = torch.arange(L, device="cuda")[None]
        hidden = key > last
        if c["window"]:
            hidden |= key <= last - c["window"]
        for g in range(Hkv):
            k, v = (torch.cat([s[x + "8"][b, :whole, g].double() *
                               s[x + "_scale"][b, :whole // T, g].double().repeat_interleave(T)[:, None],
                               s[x + "_tail"][b, :L - whole, g].double()]) for x in "kv")
            for h in range(g * H // Hkv, (g + 1) * H // Hkv):
                score = (s["q"][b, :, h].double() @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[b, h] = torch.logsumexp(score, 1)
                o[b, :, h] = torch.softmax(score, 1) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attn8 if case["op"] == "attn8" else _exact_rotary)(case, s)
