"""KVCache's checks, on the CPU: what does not fit is refused on the host,
before anything is written, and never reaches an index on the GPU."""
import pytest
import torch

from activation_compression_pamm_amd.block import KVCache


def cache(batch=3):
    c = KVCache(batch, 8, 2, 16, device="cpu", dtype=torch.float32)
    c.k.zero_()
    c.v.zero_()
    return c


def test_append():
    c = cache()
    a, b = torch.randn(3, 5, 2, 16), torch.randn(3, 5, 2, 16)
    c.append(a, b)
    c.append(a[:, :2], b[:, :2])
    assert c.used == 7 and c.lengths.tolist() == [7, 7, 7]
    assert torch.equal(c.k[:, :7], torch.cat([a, a[:, :2]], 1)) and torch.equal(c.v[:, :7], torch.cat([b, b[:, :2]], 1))


@pytest.mark.parametrize("k,v", [((1, 2, 2, 16), None), ((4, 2, 2, 16), None), ((3, 2, 1, 16), None), ((3, 2, 2, 8), None),
                                 ((3, 2, 2, 16), (3, 1, 2, 16)), ((3, 2, 2, 16), (1, 2, 2, 16)), ((3, 2, 16), None),
                                 ((3, 9, 2, 16), None)])
def test_what_does_not_fit_is_refused(k, v):
    c = cache()
    with pytest.raises(ValueError, match="KVCache"):
        c.append(torch.ones(k), torch.ones(v or k))
    assert c.used == 0 and not c.lengths.any() and not c.k.any() and not c.v.any()


def test_one_sequence_takes_no_batch():
    c = cache(1)
    with pytest.raises(ValueError, match="KVCache"):
        c.append(torch.ones(4, 2, 2, 16), torch.ones(4, 2, 2, 16))
    assert c.used == 0
    with pytest.raises(TypeError, match="KVCache"):
        c.append(torch.ones(1, 2, 2, 16).bfloat16(), torch.ones(1, 2, 2, 16).bfloat16())
    assert c.used == 0 and not c.k.any()
