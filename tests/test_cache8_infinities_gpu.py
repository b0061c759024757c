"""GPU: infinities in the values that wait in the tail of a cache in 8 bits.
What a query sees of them comes through as an infinity, as in attention();
what it does not see does not, and nothing else changes."""
import numpy as np
import pytest
import torch

import activation_compression_pamm_amd as pamm
import block_oracle as bo
from test_attention_gpu import close, dev, host, say, values
from test_cache8_gpu import BOTH, build, meant

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@BOTH
# up to 16 rows a key/value head, up to 32, more
@pytest.mark.parametrize("Sq,H,Hkv", [(1, 2, 2), (1, 16, 1), (4, 4, 1), (1, 20, 1), (8, 8, 2), (50, 2, 1)])
@pytest.mark.parametrize("L,D", [(1, 16), (31, 64), (72, 48), (200, 128)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 5)])
def test_infinities_in_the_tail(dtype, Sq, H, Hkv, L, D, causal, window):
    say("infinities in the tail", dtype, Sq, H, Hkv, L, D, causal, window)
    Sq = min(Sq, L)
    c, _, _, n = build(1, L, Hkv, D, 64, dtype, [L], [L])
    k, v = meant(c, [L], L)
    whole = L // 64 * 64
    # (token, element, value): the last token, one further back, and both signs in one element
    places = [(L - 1, 3, np.inf), (L - 1, D - 1, -np.inf), (max(L - 4, whole), 7, np.inf)]
    if L > 1:
        places += [(L - 1, 9, np.inf), (max(L - 2, whole), 9, -np.inf)]
    for at, e, x in places:
        c.v_tail[0, at - whole, 0, e] = x
        v[0, at, 0, e] = 0.0
    q = values(np.random.default_rng(1), (1, Sq, H, D), dtype)
    ref = bo.attention(q, k, v, dtype=dtype, causal=causal, window=window, kv_len=[L])
    want, sees = ref["o"], bo.visible(Sq, L, Sq, L, causal, window)
    with np.errstate(invalid="ignore"):
        for at, e, x in places:  # every probability here is far from 0
            want[0, :, :H // Hkv, e] += np.where(sees[:, at, None], x, 0.0)
    o, lse = pamm.attention_fp8(dev(q, dtype), c, n, causal=causal, window=window)
    # over attention's bounds: the values' scale is one more product of each probability
    close("o", o, want, ref["o_tol"] + 4 * bo.U * np.abs(v).max())
    close("lse", lse, ref["lse"], ref["lse_tol"])
    assert np.isposinf(host(o)[0, -1, 0, 3])
