"""The workspace of qk_norm_rotary_backward as the binding states it: enough
for every call on tensors of these shapes (no GPU needed, no kernel launched)."""
import ctypes

import pytest
import torch

import activation_compression_pamm_amd as pamm
from activation_compression_pamm_amd import position_ops as ops
from test_positions_cpu import Rotary

SIZES = [(8, 2000, 12, 12), (1, 20547, 32, 8), (3, 37, 6, 2), (1, 0, 4, 1), (2, 100000, 1, 1)]


@pytest.mark.parametrize("code,dtype,D", [(0, torch.float32, D) for D in (4, 40, 64, 68, 72, 80, 96, 128)] +
                         [(1, torch.bfloat16, D) for D in (8, 40, 64, 72, 80, 88, 96, 104, 120, 128)])
@pytest.mark.parametrize("B,S,H,Hkv", SIZES)
def test_the_size_is_enough_for_every_rotation(code, dtype, D, B, S, H, Hkv):
    """Either layout of pairs, any number of them; B, S and heads have no memory here, as sizes alone count."""
    q, k = (torch.empty(D, dtype=dtype).as_strided((B, S, h, D), (0, 0, 0, 1)) for h in (H, Hkv))
    need = [ops._lib().pamm_rotary_backward_workspace_size(ctypes.byref(Rotary(
        dtype=code, interleaved=i, batch=B, seq=S, heads_q=H, heads_k=Hkv, head_dim=D, rot_dim=r, magnitude=1.0)))
        for i in (0, 1) for r in range(0, D + 1, 2)]
    assert pamm.qk_norm_rotary_backward_workspace_size(q, k) == max(need)
