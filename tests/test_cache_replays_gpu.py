"""GPU: a captured step of the block, replayed: its tokens are the cache's, for
later replays and for calls outside the graph, without the caller's help."""
import pytest
import torch

from activation_compression_pamm_amd.block import PammAttentionBlock
from test_attention_gpu import say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("n", [1, 3])
def test_replays_and_eager_calls_between_them(eight_bits, n):
    say("replays", eight_bits, n)
    torch.manual_seed(6)
    kw = {"eight_bits": True, "block": 32} if eight_bits else {}
    block = PammAttentionBlock(128, 4, 2, rotary=True, device="cuda", dtype=torch.bfloat16).eval()
    x = torch.randn(2, 20 + 24 * n, 128, device="cuda").bfloat16()
    eager, cache, warm = (block.cache(2, 128, **kw) for _ in range(3))
    for c in (eager, cache):
        block.step(x[:, :20], None, c)
    parts = [x[:, i:i + n].clone() for i in range(20, x.shape[1], n)]
    want = [block.step(t, None, eager)[0].clone() for t in parts]
    token = parts[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(token, None, warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(token, None, cache)
    for i, t in enumerate(parts):
        if i % 8 == 5:
            got, _ = block.step(t, None, cache)
        else:
            token.copy_(t)
            graph.replay()
            got = out
        torch.cuda.synchronize()
        # the same kernels on the same keys, cut into parts elsewhere at most: 2^-8 for each of three roundings
        assert rel(got, want[i]) < 3 * 2.0 ** -8, i
        if i == 16:  # and what the cache shows by itself
            q = torch.randn(2, n, 4, 32, device="cuda").bfloat16()
            whole = block.cache(2, 128, **kw)
            block.step(x[:, :20 + 17 * n], None, whole)
            assert rel(cache.attend(q), whole.attend(q)) < 3 * 2.0 ** -8
    assert cache.lengths.tolist() == [x.shape[1]] * 2 == eager.lengths.tolist()
    with pytest.raises(ValueError, match="do not fit"):
        block.step(torch.zeros(2, 129 - x.shape[1], 128, device="cuda").bfloat16(), None, cache)


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("n", [1, 3])
def test_replays_past_the_room_drop_their_tokens(eight_bits, n):
    """Sequences of different lengths, the longer of which is full first; nothing behind the room is written."""
    say("replays past the room", eight_bits, n)
    room, start, calls = 40, 29, 14
    block = PammAttentionBlock(64, 2, 1, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(2, start + calls * n, 1, 32, device="cuda", generator=g).bfloat16() for _ in "kv")
    cache, want, warm = (block.cache(2, room, **({"eight_bits": True, "block": 32} if eight_bits else {})) for _ in range(3))
    cache.append(k[:, :start], v[:, :start])
    cache.lengths[1] -= 5  # the second sequence takes its last tokens back
    token = [t[:, :n].clone() for t in (k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.append(*token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(*token)
    for i in range(calls):
        for t, x in zip(token, (k, v)):
            t.copy_(x[:, start + i * n:start + (i + 1) * n])
        graph.replay()
    torch.cuda.synchronize()
    lengths = [min(start + calls * n, room), min(start - 5 + calls * n, room)]
    assert cache.lengths.tolist() == lengths
    m = min(lengths)
    want.append(*(torch.stack([x[0, :m], torch.cat([x[1, :start - 5], x[1, start:]])[:m]]) for x in (k, v)))
    if eight_bits:
        whole = m // 32 * 32
        for a, b in zip(cache.tensors, want.tensors):
            top = whole if a.dtype == torch.float8_e4m3fn else whole // 32 if a.dtype == torch.float32 else m - whole
            assert torch.equal(a[:, :top].float(), b[:, :top].float())
    else:
        assert torch.equal(cache.k[:, :m], want.k[:, :m]) and torch.equal(cache.v[:, :m], want.v[:, :m])
