"""Groups that several CTAs share, call after call on one workspace: every row is written, and to the same bits."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_cut_groups_of_calls_that_follow_one_another(dtype):
    """One to eight long groups (a CTA's shares), and 40 (a warp's), of the tree and of lists, in turn."""
    rng = np.random.default_rng(3)
    hkv, d, nb, width = 2, 128, 4200, 1024
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    pool = ref.random_pool(pkv.Pool(nb, hkv, d, **kw), 3)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, 1)
    calls = []
    for n, blocks in ((1, 1024), (2, 700), (4, 1000), (20, 200)):
        bt = ref.dev(ref.tables(rng, [blocks * 16] * n, nb, width))
        ctx = ref.dev(np.full(n, blocks * 16, np.int32))
        cu = ref.dev(np.arange(n + 1).astype(np.int32))
        pos = ref.dev(np.full(n, blocks * 16 - 1, np.int32))
        q = torch.randn((n, 8, d), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
        mask = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
        sel = ref.dev(np.tile(np.arange(blocks, dtype=np.int32), (n, hkv, 1)))
        o, lse = torch.empty_like(q), torch.empty((n, 8), device="cuda")
        calls.append((lambda bt=bt, ctx=ctx, cu=cu, q=q, mask=mask, o=o, lse=lse:
                      pkv.pkv_tree_attn(pool, q, bt, ctx, ctx - 9, cu, mask, 0.1, out=o, lse=lse), o, lse))
        o, lse = torch.empty_like(q), torch.empty((n, 8), device="cuda")
        calls.append((lambda bt=bt, cu=cu, q=q, pos=pos, sel=sel, o=o, lse=lse:
                      pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1, out=o, lse=lse), o, lse))
    want = []
    for call, o, lse in calls:
        call()
        torch.cuda.synchronize()
        want.append((o.clone(), lse.clone()))
    # The tree's prefix and last nine slots are all blocks' keys: the two LSEs are off by ds each (attn_ref), with
    # B <= scale |q| |k| <= 0.1 * 17 * 17 (norms of 128 normal values; FP8 keys have that size too).
    ds = (d + 8) * 2.0 ** -24 * 0.1 * 17 * 17 + 2.0 ** -15
    for a, b in zip(want[::2], want[1::2]):
        la, lb = (x[1].double().cpu().numpy() for x in (a, b))
        ref.assert_close(la, lb, np.full(la.shape, 2 * ds + 2.0 ** -24 * np.abs(lb).max()), "LSE")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        for _, o, lse in calls:
            o.fill_(7.0)
            lse.fill_(7.0)
        for call, _, _ in calls:                        # back to back: one workspace, no wait between them
            call()
        for (_, o, lse), (wo, wl) in zip(calls, want):
            differ += (o != wo).sum() + (lse != wl).sum()
    assert int(differ) == 0
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()
