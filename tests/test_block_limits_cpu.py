"""Limits of the block operators' C ABI, on the host (no kernel is launched)."""
import ctypes

import pytest

from activation_compression_pamm_amd import block_ops as ops
from test_block_abi_cpu import ESHAPE, FAKE, problem


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


ONE = ops._Heads(FAKE, 64, 64, 64)
# workgroups of 256 threads: heads x tiles of 128 rows; a grid holds less than 2^32 threads
FORWARD = [dict(batch=2**24, heads=1, heads_kv=1, seq_q=1, seq_k=1), dict(batch=2**17, heads=128, heads_kv=128, seq_q=1, seq_k=1),
           dict(batch=2**21, heads=8, heads_kv=1, seq_q=128, seq_k=1)]
BACKWARD = FORWARD + [dict(batch=2**17, heads=1, heads_kv=1, seq_q=1, seq_k=128 * 127),
                      dict(batch=2**23, heads=1, heads_kv=1, seq_q=128, seq_k=1)]


def tight(**kw):
    p = problem(head_dim=8, tensors={n: ONE for n in "qkvo"}, **kw)
    return ctypes.byref(p)


@pytest.mark.parametrize("sizes", range(len(FORWARD)))
def test_more_workgroups_than_a_grid_holds(lib, sizes):
    assert lib.pamm_attention_workspace_size(tight(**FORWARD[sizes])) == 0
    assert lib.pamm_attention(tight(**FORWARD[sizes]), FAKE, 1 << 62, None) == ESHAPE


@pytest.mark.parametrize("sizes", range(len(BACKWARD)))
def test_more_workgroups_than_the_backward_pass_s_grids_hold(lib, sizes):
    p, h = tight(**BACKWARD[sizes]), ctypes.byref(ONE)
    assert lib.pamm_attention_backward_workspace_size(p) == 0
    assert lib.pamm_attention_backward(p, h, h, h, h, FAKE, 1 << 62, None) == ESHAPE


def test_sizes_below_the_limits_have_workspaces(lib):
    assert lib.pamm_attention_backward_workspace_size(tight(batch=2**22, heads=1, heads_kv=1, seq_q=128, seq_k=128)) > 2**31
    assert lib.pamm_attention_backward_workspace_size(tight(batch=1, heads=1, heads_kv=1, seq_q=2**20, seq_k=2**29)) > 0
