"""Plain 64-bit definitions of the rotation of queries and keys and of their
norm, and how far a kernel with 32-bit sums may be from them, element by
element.

Rounding model as in block_oracle: u = 2^-24, r the output type's, gamma_m for
a sum of m products.  A cosine or sine is off by at most 4 u: the reduced
angle (at most pi / 4) is rounded once, the series' last steps are, and what
they add to is at most 1; p * inv_freq itself, in 64 bits, by 2^-51 of the
angle.  With magnitude m (one more rounding) and n the row before its
rotation, off by E_n relative,

    y:   m (5 u + |angle| 2^-51 + 2 u + E_n) (|n_a| + |n_b|) + r |y|

E_n is 0 without a norm, else E = gamma_D + 8 u (rstd) and 2 u for the two
products.  Backward, with e_g the first two terms of that for g (from dy):

    u = g w:    e_u = e_g |w| + u |u|
    mean(u xhat): e_m = mean(e_u |xhat|) + (E + gamma_D + 4 u) mean |u xhat|
    dx: rstd (e_u + |xhat| e_m + (2 E + 4 u) (|u| + |xhat mean|)) + r |dx|
    dw: sum e_g |xhat| + (E + 2 u + gamma_N) sum |g xhat|,  N tokens x heads.
"""
import numpy as np

from block_oracle import R, U, gamma


def angles(positions, inv_freq):
    """[B, S] and [R / 2] -> [B, S, 1, R / 2]"""
    return np.asarray(positions, np.float64)[:, :, None, None] * np.asarray(inv_freq, np.float64)


def split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def joined(a, b, x, rot, interleaved):
    y = x.copy()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


def rotate(x, t, *, interleaved=False, magnitude=1.0, inverse=False, E=0.0):
    """x [B, S, H, D]; returns (y, what it may be off by before its rounding)."""
    rot = 2 * t.shape[-1]
    a, b = split(x, rot, interleaved)
    c, s = np.cos(t), np.sin(-t if inverse else t)
    y = joined(magnitude * (a * c - b * s), magnitude * (a * s + b * c), x, rot, interleaved)
    with np.errstate(invalid="ignore"):
        off = abs(magnitude) * (7 * U + np.abs(t) * 2.0 ** -51 + E) * (np.abs(a) + np.abs(b))
    return y, joined(off, off, E * np.abs(x), rot, interleaved)


def rotary(x, positions, inv_freq, *, dtype="f32", **kw):
    y, off = rotate(x, angles(positions, inv_freq), **kw)
    return y, off + R[dtype] * np.abs(y)


def norm_rotary(x, w, positions, inv_freq, *, eps=1e-6, dy=None, dtype="f32", **kw):
    """One of q and k: {"y", "y_tol"} and with dy also dx and dw."""
    D, r, t = x.shape[-1], R[dtype], angles(positions, inv_freq)
    E = gamma(D) + 8 * U
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    y, off = rotate(xhat * w, t, E=E + 2 * U, **kw)
    res = {"y": y, "y_tol": off + r * np.abs(y)}
    if dy is not None:
        g, eg = rotate(dy, t, inverse=True, **kw)
        u = g * w
        eu = eg * np.abs(w) + U * np.abs(u)
        mean = (u * xhat).mean(-1, keepdims=True)
        em = (eu * np.abs(xhat)).mean(-1, keepdims=True) + (E + gamma(D) + 4 * U) * np.abs(u * xhat).mean(-1, keepdims=True)
        res["dx"] = rstd * (u - xhat * mean)
        res["dx_tol"] = rstd * (eu + np.abs(xhat) * em + (2 * E + 4 * U) * (np.abs(u) + np.abs(xhat * mean))) + r * np.abs(res["dx"])
        n = int(np.prod(x.shape[:-1]))
        res["dw"] = (g * xhat).sum((0, 1, 2))
        res["dw_tol"] = (eg * np.abs(xhat)).sum((0, 1, 2)) + (E + 2 * U + gamma(n)) * np.abs(g * xhat).sum((0, 1, 2))
    return res
