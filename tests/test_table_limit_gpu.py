"""The widest table: key positions, rounded up to a key tile, have to stay below 2^31."""
import ctypes

import pytest
import torch

from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_tables_beyond_the_limit_are_refused():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pool, lib, n = pkv.Pool(4, 1, 64), pkv.load_library(), ctypes.c_size_t()
    most = (2 ** 31 - 1 - 128) // 16
    assert lib.pkv_select_blocks_workspace_size(pool.handle, most, 1, ctypes.byref(n)) == pkv.PKV_OK
    p = pool.k.data_ptr()
    for width in (most + 1, 2 ** 27 - 2, 2 ** 27, 2 ** 31 - 1):      # refused before anything is read
        h = pool.handle
        assert lib.pkv_select_blocks_workspace_size(h, width, 1, ctypes.byref(n)) == pkv.PKV_EINVAL
        assert lib.pkv_tree_attn(h, p, 1, p, width, p, p, p, 1, 1, p, 1, 0.1, p, None, p, 1 << 40, None) == pkv.PKV_EINVAL
        assert lib.pkv_summarize(h, p, width, 1, p, p, p, 1, p, p, None) == pkv.PKV_EINVAL
        assert lib.pkv_select_blocks(h, p, 1, p, p, width, p, 1, 1, p, p, 1, 0, 0, p, p, 1 << 40, None) == pkv.PKV_EINVAL
        assert lib.pkv_sparse_attn(h, p, 1, p, p, width, p, 1, 1, p, 1, 0.1, p, None, p, 1 << 40, None) == pkv.PKV_EINVAL
        assert lib.pkv_fork(h, p, 1, width, p, p, p, p, 1, p, p, p, None, None, p, 1 << 40, None) == pkv.PKV_EINVAL
        assert lib.pkv_compact(h, p, width, 1, p, p, p, 1, None) == pkv.PKV_EINVAL
    pool.close()
