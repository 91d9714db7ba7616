"""Which form a small batch's groups take on the rows kernel, seen from its launches: whole groups need no merge."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


def merges(ctxs, hq=64, hkv=8):
    """Merge launches for one token a request; the outputs are checked."""
    pool = ref.random_pool(pkv.Pool(sum((c + 15) // 16 for c in ctxs) + 1, hkv, 128), 1)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, 1)
    n = len(ctxs)
    ctx = np.array(ctxs, np.int32)
    bt = ref.tables(np.random.default_rng(1), ctx, pool.num_blocks)
    cu = np.arange(n + 1).astype(np.int32)
    q = torch.randn((n, hq, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    mask = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pkv.pkv_profile_enable(pool, True)
    o, lse = pkv.pkv_tree_attn(pool, q, ref.dev(bt), ref.dev(ctx), ref.dev(ctx - 1), ref.dev(cu), mask, 0.1)
    torch.cuda.synchronize()
    got = pkv.pkv_profile_read(pool, reset=True)
    pkv.pkv_profile_enable(pool, False)
    assert got["split_kv"]["launches"] == 1
    K, V = ref.pool_values(pool, "k"), ref.pool_values(pool, "v")
    for r in range(n):
        for g in range(hkv):
            k, _ = ref.gather(K, bt[r], ctxs[r], g)
            v, _ = ref.gather(V, bt[r], ctxs[r], g)
            G = hq // hkv
            rows = q[r, g * G:(g + 1) * G].double().cpu().numpy()
            want, wl, to, tl = ref.softmax_rows(rows, k, v, np.ones((G, ctxs[r]), bool), 0.1, False)
            ref.assert_close(o[r, g * G:(g + 1) * G].float().cpu().numpy(), want, to, "O")
            ref.assert_close(lse[r, g * G:(g + 1) * G].cpu().numpy(), wl, tl, "LSE")
    pool.close()
    return got["merge"]["launches"]


def test_one_long_request_among_short_ones_is_shared_out():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert merges([6000] + [300] * 11) == 1               # 375 blocks: its groups would be waited for
    assert merges([2000] + [300] * 11) == 0               # 125 blocks: no merge is worth more
    assert merges([6000], hq=16, hkv=2) == 1              # one request: equal groups, far fewer than SMs
    assert merges([1500], hq=16, hkv=2) == 0
