"""Plain 64-bit definitions of the operators around the projection, and how
far a kernel with 32-bit sums may be from them, element by element.

Rounding model.  u = 2^-24 is fp32's unit roundoff, r the output type's (2^-8
for bf16, u for fp32).  A sum of m fp32 products is off by at most
gamma_m = m u / (1 - m u) times the sum of the products' absolute values
(Higham, Accuracy and Stability of Numerical Algorithms, section 3.1).

Attention.  A score is off by E_s = gamma_D * scale * max sum|q k| plus the
rounding of its scaling and of the exponent (4 u max(|s|, 1), log2 units
included); a probability is then off by a factor within 1 +- E,
E = 4 (E_s + gamma_S + 4 u): numerator, sum and lse.  With A = the same sum
over absolute values as the result's, results are within

    o:   (E + rp) sum P|v| + r|o|          rp = r: P is rounded to bf16 once
    dv:  (E + rp) sum P|do| + r|dv|
    delta: its o is rounded (r sum|do||o|) and summed (gamma_D sum|do||o|)
    dS:  E |dS| + P (|d delta| + gamma_D sum|do||v|), then rounded (rp |dS|)
    dq:  scale (d dS |k|) + gamma_S scale |dS||k| + r|dq|,  dk alike.
"""
import numpy as np

U = 2.0 ** -24
R = {"bf16": 2.0 ** -8, "f32": U}


def gamma(m):
    return m * U / (1 - m * U)


def visible(Sq, Sk, Lq, Lk, causal, window):
    i, j = np.arange(Sq)[:, None], np.arange(Sk)[None]
    m = (i < Lq) & (j < Lk)
    if causal:
        m &= j <= i + Lk - Lq
        if window:
            m &= j > i + Lk - Lq - window
    return m


def attention(q, k, v, do=None, *, causal=False, window=0, scale=None, q_len=None, kv_len=None, dtype="f32"):
    """q [B, Sq, H, D], k, v [B, Sk, Hkv, D] float64.  Returns a dict of
    results and, under "<name>_tol", their elementwise bounds."""
    B, Sq, H, D = q.shape
    Sk, Hkv = k.shape[1:3]
    G = H // Hkv
    scale = 1 / np.sqrt(D) if scale is None else scale
    r, rp = R[dtype], (R[dtype] if dtype == "bf16" else 0.0)
    z = np.zeros
    res = {"o": z(q.shape), "lse": np.full((B, H, Sq), -np.inf), "o_tol": z(q.shape), "lse_tol": z((B, H, Sq))}
    if do is not None:
        res |= {n + t: z(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v)) for t in ("", "_tol")}
    for b in range(B):
        Lq = Sq if q_len is None else int(np.clip(q_len[b], 0, Sq))
        Lk = Sk if kv_len is None else int(np.clip(kv_len[b], 0, Sk))
        m = visible(Sq, Sk, Lq, Lk, causal, window)
        seen = m.any(1)
        if not seen.any():
            continue
        for h in range(H):
            g = h // G
            # what the mask hides takes no part, whatever it holds
            Q, K, V = q[b, :, h], np.where(m.any(0)[:, None], k[b, :, g], 0.0), np.where(m.any(0)[:, None], v[b, :, g], 0.0)
            Q = np.where(seen[:, None], Q, 0.0)
            s = np.where(m, scale * (Q @ K.T), -np.inf)
            top = np.where(seen, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - top[:, None])
            tot = e.sum(1)
            P = e / np.where(tot > 0, tot, 1.0)[:, None]
            lse = np.where(seen, top + np.log(np.where(tot > 0, tot, 1.0)), -np.inf)
            absqk = abs(scale) * (np.abs(Q) @ np.abs(K).T).max(initial=0.0)
            E = 4 * (gamma(D) * absqk + 4 * U * max(absqk, 1.0) + gamma(Sk) + 4 * U)
            o = P @ V
            res["o"][b, :, h], res["lse"][b, h] = o, lse
            res["o_tol"][b, :, h] = (E + rp) * (P @ np.abs(V)) + r * np.abs(o)
            res["lse_tol"][b, h] = E + 4 * U * np.abs(np.where(seen, lse, 0.0))
            if do is None:
                continue
            dO = np.where(seen[:, None], do[b, :, h], 0.0)
            dP, delta = dO @ V.T, (dO * o).sum(1)
            dS = np.where(m, P * (dP - delta[:, None]), 0.0)
            ado = (np.abs(dO) * (np.abs(o) + res["o_tol"][b, :, h])).sum(1)
            d_delta = (np.abs(dO) * res["o_tol"][b, :, h]).sum(1) + (r + gamma(D)) * ado
            d_dS = (E + rp) * np.abs(dS) + P * (d_delta[:, None] + gamma(D) * (np.abs(dO) @ np.abs(V).T))
            d_dS = d_dS * (1 + rp) + gamma(Sk) * np.abs(dS)
            Kz, aK, aQ = K, np.abs(K), np.abs(Q)
            res["dq"][b, :, h] = scale * (dS @ Kz)
            res["dq_tol"][b, :, h] = abs(scale) * (d_dS @ aK) + r * np.abs(res["dq"][b, :, h])
            res["dk"][b, :, g] += scale * (dS.T @ Q)
            res["dk_tol"][b, :, g] += abs(scale) * ((d_dS + gamma(Sq * G) * np.abs(dS)).T @ aQ)
            res["dv"][b, :, g] += P.T @ dO
            res["dv_tol"][b, :, g] += (E + rp + gamma(Sq * G)) * (P.T @ np.abs(dO))
    if do is not None:
        for n in ("dk", "dv"):
            res[n + "_tol"] += r * np.abs(res[n])
    return res


def to_bf16(x):
    """float64 -> the nearest bf16 value (through fp32 first, as the kernels do), as float64."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return u.view(np.float32).astype(np.float64)


def e4m3(x):
    """The nearest 8-bit float (4 exponent, 3 fraction bits, largest 448), ties to even."""
    a = np.abs(x)
    unit = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.clip(np.round(x / unit) * unit, -448, 448)


def add_rms_norm(x, w, r=None, *, eps=1e-6, dtype="f32", dy=None, dh=None):
    """x, r, dy, dh [n, d] and w [d], float64 holding values of the dtype.
    rstd is off by gamma_d (sum of squares) and a few roundings, y by that and
    three more, then rounded; dx's terms are products of up to five such
    factors around one sum of d terms."""
    d = x.shape[1]
    ro = R[dtype]
    h = x if r is None else (to_bf16(x + r) if dtype == "bf16" else (x + r).astype(np.float32).astype(np.float64))
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    E = gamma(d) + 8 * U
    xhat = h * rstd[:, None]
    y = xhat * w
    res = {"h": h, "rstd": rstd, "rstd_tol": E * rstd, "y": y, "y_tol": (E + 4 * U + ro) * np.abs(y)}
    scale = np.maximum(np.abs(y).max(1) / 448, 2.0 ** -126)
    res |= {"scale": scale, "scale_tol": (E + 8 * U) * scale}
    if dy is not None:
        g = dy * w
        mean = (g * xhat).mean(1, keepdims=True)
        dx = rstd[:, None] * (g - xhat * mean) + (0 if dh is None else dh)
        mean_tol = (2 * E + gamma(d) + 8 * U) * (np.abs(g * xhat)).mean(1, keepdims=True)
        size = rstd[:, None] * (np.abs(g) + np.abs(xhat * mean)) + (0 if dh is None else np.abs(dh))
        res["dx"], res["dx_tol"] = dx, (2 * E + 8 * U) * size + rstd[:, None] * np.abs(xhat) * mean_tol + ro * np.abs(dx)
        res["dw"] = (dy * xhat).sum(0)
        res["dw_tol"] = (E + 4 * U + gamma(x.shape[0])) * np.abs(dy * xhat).sum(0)
    return res
