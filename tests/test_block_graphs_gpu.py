"""GPU: the block's operators in a captured graph, replayed on new inputs, with
eager work of the same operators and of others between the replays."""
import pytest
import torch

import activation_compression_pamm_amd as pamm
from test_attention_gpu import say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def operators():
    """name -> (inputs, call on them)"""
    g = torch.Generator(device="cuda").manual_seed(17)

    def r(*s, dtype=torch.bfloat16):
        return torch.randn(*s, generator=g, device="cuda").to(dtype)

    n = torch.tensor([900, 17], dtype=torch.int32, device="cuda")

    def step(q, k, v, do):
        o, lse = pamm.attention(q, k, v, causal=True, window=200)
        return (o, lse, *pamm.attention_backward(do, q, k, v, o, lse, causal=True, window=200))

    def norm(x, res, w, dy):
        y, h, rstd = pamm.add_rms_norm(x, w, res)
        q, scale, _, _ = pamm.add_rms_norm_fp8(x, w, res)
        return (y, h, q.float(), scale, *pamm.add_rms_norm_backward(dy, h, w, rstd, dh=h))

    def clip(a, b):
        out = [torch.empty_like(a), torch.empty_like(b)]
        return (pamm.clip_grad_norm([a, b], 1.0, out=out), *out)

    return {"token": ((r(2, 1, 8, 64), r(2, 900, 2, 64), r(2, 900, 2, 64)),
                      lambda q, k, v: pamm.attention(q, k, v, causal=True, kv_len=n)),
            "chunk": ((r(2, 60, 8, 64), r(2, 900, 2, 64), r(2, 900, 2, 64)),
                      lambda q, k, v: pamm.attention(q, k, v, causal=True)),
            "step": ((r(2, 300, 4, 64), r(2, 300, 2, 64), r(2, 300, 2, 64), r(2, 300, 4, 64)), step),
            "long step": ((r(1, 1100, 16, 128), r(1, 1100, 16, 128), r(1, 1100, 16, 128), r(1, 1100, 16, 128)), step),
            "norm": ((r(500, 768), r(500, 768), r(768), r(500, 768)), norm),
            "clip": ((r(3000, 30, dtype=torch.float32), r(701)), clip)}


@pytest.mark.parametrize("name", ["token", "chunk", "step", "long step", "norm", "clip"])
def test_replays_are_the_eager_results(name):
    say("graph", name)
    inputs, call = operators()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*inputs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*inputs)
    for i in range(4):
        for t in inputs:
            t.mul_(1.25 if i % 2 else -0.75)
        if name == "step" and i == 2:
            inputs[2][0, 250] = float("nan")  # marks work for the second pass
        want = call(*inputs)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0)), i
        if name == "step" and i == 2:
            assert torch.isnan(got[0]).any()
            inputs[2].nan_to_num_(0.5)
