"""GPU: the block's operators on a stream other than the current one."""
import pytest
import torch

import activation_compression_pamm_amd as pamm
from test_attention_gpu import say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def calls():
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()

    q, k, v, do = r(2, 300, 4, 64), r(2, 900, 2, 64), r(2, 900, 2, 64), r(2, 300, 4, 64)
    o, lse = pamm.attention(q, k, v, causal=True)
    x, w, dy = r(500, 768), r(768), r(500, 768)
    _, h, rstd = pamm.add_rms_norm(x, w, dy)
    big = [r(1000, 300), r(77)]
    return {
        "attention": lambda s: pamm.attention(q, k, v, causal=True, stream=s),
        "attention_backward": lambda s: pamm.attention_backward(do, q, k, v, o, lse, causal=True, stream=s),
        "add_rms_norm": lambda s: pamm.add_rms_norm(x, w, dy, stream=s),
        "add_rms_norm_fp8": lambda s: pamm.add_rms_norm_fp8(x, w, dy, stream=s),
        "add_rms_norm_backward": lambda s: pamm.add_rms_norm_backward(dy, h, w, rstd, dh=x, stream=s),
        "clip_grad_norm": lambda s: (pamm.clip_grad_norm(big, stream=s),),
    }


@pytest.mark.parametrize("name", ["attention", "attention_backward", "add_rms_norm", "add_rms_norm_fp8",
                                  "add_rms_norm_backward", "clip_grad_norm"])
def test_results_and_memory_belong_to_the_stream(name):
    """Results are those of the current stream, also while that one allocates and
    overwrites whatever it may take, and what the call allocates is the side
    stream's: blocks freed on the current stream, whose pending work may still
    use them, are not written."""
    say("stream", name)
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        freed = [torch.empty_like(t) for t in want]
        mine = {t.untyped_storage().data_ptr() for t in freed}
        del freed  # now the current stream's to give
        got = call(side)
        assert not mine & {t.untyped_storage().data_ptr() for t in got}
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 22)]
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8) if a.dim() else a, b.view(torch.uint8) if b.dim() else b)
        del junk
