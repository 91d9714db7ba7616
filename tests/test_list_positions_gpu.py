"""Attention over lists: positions outside the table are flagged; below 0 no key is seen, beyond it all of the blocks'."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("p,flag", [(0, False), (95, False), (96, True), (2 ** 31 - 1, True), (-1, True), (-2 ** 31, True)])
def test_positions_around_the_table(p, flag, dtype):
    from paged_kv_attention_25_gb300 import build
    build.build()
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    pool = ref.random_pool(pkv.Pool(8, 2, 64, **kw), 1)
    bt = np.array([[5, 2, 7, 0, 1, 6]], np.int32)
    q = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    lists = np.tile(np.array([3, 0, 5, -1, 1, 2, 4], np.int32), (1, 2, 1))
    o, lse = pkv.pkv_sparse_attn(pool, q, ref.dev(np.array([p], np.int32)), ref.dev(bt), ref.dev(np.array([0, 1], np.int32)),
                                 ref.dev(lists), 0.1)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(pool) == (pkv.PKV_DEVERR_POSITION if flag else 0)
    K, V = ref.pool_values(pool, "k"), ref.pool_values(pool, "v")
    for g in range(2):
        k, _ = ref.gather(K, bt[0], 96, g)
        v, _ = ref.gather(V, bt[0], 96, g)
        rows = q[0, 2 * g:2 * g + 2].double().cpu().numpy()
        want, wl, to, tl = ref.softmax_rows(rows, k, v, np.repeat(np.arange(96)[None] <= p, 2, 0), 0.1, dtype != "bf16")
        ref.assert_close(o[0, 2 * g:2 * g + 2].float().cpu().numpy(), want, to, "O")
        ref.assert_close(lse[0, 2 * g:2 * g + 2].cpu().numpy(), wl, tl, "LSE")
    pool.close()
