"""Refusals of the tree attention, the block-selected attention and the page calls: host checks, no GPU."""
import ctypes

import pytest
import torch

from paged_kv_attention_25_gb300 import build as pkv_build
from paged_kv_attention_25_gb300 import pkv


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def test_null_pool(lib):
    n = ctypes.c_size_t()
    assert lib.pkv_tree_mask(None, None, None, 1, 1, None, 1, None) == pkv.PKV_EINVAL
    assert lib.pkv_tree_attn_workspace_size(None, 8, 1, 1, 1, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_tree_attn(None, None, 8, None, 1, None, None, None, 1, 1, None, 1, 1.0, None, None, None, 0,
                             None) == pkv.PKV_EINVAL
    assert lib.pkv_summarize(None, None, 1, 1, None, None, None, 1, None, None, None) == pkv.PKV_EINVAL
    assert lib.pkv_select_blocks_workspace_size(None, 1, 1, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_select_blocks(None, None, 8, None, None, 1, None, 1, 1, None, None, 1, 0, 0, None, None, 0,
                                 None) == pkv.PKV_EINVAL
    assert lib.pkv_sparse_attn_workspace_size(None, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_sparse_attn(None, None, 8, None, None, 1, None, 1, 1, None, 1, 1.0, None, None, None, 0,
                               None) == pkv.PKV_EINVAL
    assert lib.pkv_fork_workspace_size(None, 1, 1, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_fork(None, None, 0, 1, None, None, None, None, 0, None, None, None, None, None, None, 0,
                        None) == pkv.PKV_EINVAL
    assert lib.pkv_copy_blocks(None, None, None, 1, None, None, None) == pkv.PKV_EINVAL
    assert lib.pkv_compact(None, None, 1, 1, None, None, None, 1, None) == pkv.PKV_EINVAL
    assert "pool" in pkv.pkv_last_error()


class FakePool:
    """Stands in for a pool in the wrapper's own checks, which come before the library is called."""

    def __init__(self):
        self.k = torch.zeros(1)
        self.num_blocks, self.num_kv_heads, self.head_dim = 8, 2, 64
        self.handle, self.device_index = None, 0


I1, I2, Q = torch.zeros(3, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32), torch.zeros((2, 2, 64), dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda p: pkv.pkv_tree_attn(p, Q, I2, I1, I1, I1, I2, 1.0),
    lambda p: pkv.pkv_tree_mask(p, I1, I1),
    lambda p: pkv.pkv_select_blocks(p, None, Q, I1, I2, I1, 4),
    lambda p: pkv.pkv_sparse_attn(p, Q, I1, I2, I1, Q, 1.0),
    lambda p: pkv.pkv_summarize(p, None, I2, I1, I1, I1),
    lambda p: pkv.pkv_fork(p, I2, I1, I1, I1, I1, I1),
    lambda p: pkv.pkv_copy_blocks(p, I1, I1),
    lambda p: pkv.pkv_compact(p, I2, I1, I1, I1),
    lambda p: pkv.BlockSummary(p, Q, Q),
    lambda p: pkv.pkv_compact(p, [[0]], [0, 1], [0], [0]),
])
def test_tensors_that_are_not_on_the_device_are_refused(call):
    with pytest.raises(TypeError, match="CUDA tensor"):
        call(FakePool())


@pytest.mark.parametrize("call", [
    lambda p: pkv.pkv_tree_attn(p, Q, I1, I1, I1, I1, I2, 1.0),
    lambda p: pkv.pkv_fork(p, I1, I1, I1, I1, I1, I1),
    lambda p: pkv.pkv_copy_blocks(p, I2, I1),
])
def test_wrong_dimensions_are_refused(call):
    with pytest.raises(ValueError, match="dimensions"):
        call(FakePool())
