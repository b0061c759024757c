"""Plain 64-bit definition of a cache in 8 bits: what it holds of its tokens.

Values are e4m3(448 x / max|x|) over a block of tokens of one head.  For bf16
tokens (8 bits each) the quotient of 7 x and max|x| is no closer to a tie of
the 8-bit type (5 bits) than 2^-13 of it unless it is one, so 32 bits with a
correction round as the definition does, ties to even included: equality.
Tokens in 32 bits have quotients as near to a tie as 2^-25; the kernel's is
off by 4 u at most, and where the definition's lies within that of a tie
either neighbour is right.  Scales are one correctly rounded division.
"""
import numpy as np

from block_oracle import U, e4m3


def blocks(x, block):
    """x [S, H, D] -> (values [S', H, D], scales [S' / block, H]) of the whole blocks."""
    S = x.shape[0] // block * block
    y = x[:S].reshape(-1, block, *x.shape[1:])
    size = np.where(np.isfinite(y), np.abs(y), 0.0).max((1, 3), initial=0.0)
    size = np.maximum(size, 448 * 2.0 ** -126)
    # 448 x is exact, so that a quotient which is a tie is one here too
    q = np.where(np.isfinite(y), e4m3(448 * np.where(np.isfinite(y), y, 0.0) / size[:, None, :, None]), np.nan)
    return q.reshape(S, *x.shape[1:]), size / 448


def near_tie(x, block):
    """Whether each x / scale is within 4 u of the middle of two 8-bit values."""
    S = x.shape[0] // block * block
    y = x[:S].reshape(-1, block, *x.shape[1:])
    v = 448 * np.abs(y) / np.maximum(np.abs(y).max((1, 3)), 448 * 2.0 ** -126)[:, None, :, None]
    unit = np.exp2(np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3)
    return (np.abs(v / unit - np.floor(v / unit) - 0.5) <= 4 * U * v / unit).reshape(S, *x.shape[1:])
