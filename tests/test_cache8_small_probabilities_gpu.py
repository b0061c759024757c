"""GPU: attention over a cache in 8 bits where one key takes nearly all of the
weight, but has values of 0: the results are what the many others leave, and
have to be as exact in relation to that as any other result."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import close, dev, lens, say, values
from test_cache8_gpu import BOTH, filled, meant, rounded

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def attend(dtype, Sq, G, L, below, sink, large, spread, window=0, block=32, D=32):
    """The key `sink` scores `below` nats more than the others, whose scores spread by `spread`; the values of the
    block at `large` are 1000 times the others', and its keys score another 30 nats less."""
    say("small probabilities", dtype, Sq, G, L, below, sink, large, spread, window)
    rng = np.random.default_rng(7)
    k, v = values(rng, (L, 1, D), dtype) * spread, values(rng, (L, 1, D), dtype) + 0.5
    k[:, :, 0], k[sink, :, 0], v[sink] = 0.0, below, 0.0
    if large is not None:
        at = slice(large, large + block)
        v[at] *= 1000.0
        k[at, :, 0] = -30.0
    k, v = rounded([k, v], dtype)
    q = values(rng, (1, Sq, G, D), dtype) * 0.25
    q[..., 0] = 1.0
    c, n = filled(1, L, 1, D, block, dtype), lens([0])
    pamm.cache_append_fp8(c, dev(k[None], dtype), dev(v[None], dtype), n)
    k, v = meant(c, [L], L)
    kw = dict(causal=True, window=window, scale=1.0)
    ref = bo.attention(q, k, v, dtype=dtype, kv_len=[L], **kw)
    o, lse = pamm.attention_fp8(dev(q, dtype), c, n, **kw)
    # one more product for each probability: 4 u of a row's sum of P |v|, which the bound's P part holds 2^-8 or
    # E >= 16 u of.  No absolute term: all of a row's sum may be small
    close("o", o, ref["o"], 1.5 * ref["o_tol"])
    close("lse", lse, ref["lse"], ref["lse_tol"])


@BOTH
@pytest.mark.parametrize("Sq,G", [(1, 2), (1, 32), (33, 1), (130, 2)])
@pytest.mark.parametrize("below", [8.0, 14.5, 22.0, 40.0, 70.0])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_a_key_that_draws_attention(dtype, Sq, G, below, spread):
    """With equal scores behind it every probability is rounded in the same direction."""
    attend(dtype, Sq, G, 4096 + 17, below, 0, None, spread)


@BOTH
@pytest.mark.parametrize("Sq,G", [(1, 2), (1, 32), (130, 2)])
@pytest.mark.parametrize("below", [0.0, 9.0, 20.0])
@pytest.mark.parametrize("sink,large", [(0, 64), (2100, 64), (0, 4000)])
def test_beside_large_values(dtype, Sq, G, below, sink, large):
    attend(dtype, Sq, G, 4096, below, sink, large, 1.0)


@pytest.mark.parametrize("below", [14.0, 14.5, 25.0])
def test_a_long_tail(below):
    attend("bf16", 40, 1, 131072, below, 0, None, 0.0)


@BOTH
def test_large_values_before_the_window(dtype):
    """Nobody sees them, but they lie in a tile's reach of what is seen."""
    attend(dtype, 130, 1, 2048, 12.0, 2048 - 140, 1024, 1.0, window=1000)
