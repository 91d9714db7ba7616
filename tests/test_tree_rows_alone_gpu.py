"""A request's rows of the tree attention depend on its own inputs alone, bit for bit: not on the queries of the requests
beside it, and not on what the calls before left in the kernel's shared memory."""
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


def batch(pool, seed, prefix, nodes, hq, form):
    """A call of the tree attention on random trees; the queries are its argument."""
    rng = np.random.default_rng(seed)
    prefix = np.array(prefix, np.int32)
    ctx = (prefix + nodes).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    bt = ref.dev(ref.tables(rng, ctx, pool.num_blocks))
    mask = ref.dev(rng.integers(-2 ** 31, 2 ** 31, (int(cu[-1]), (max(nodes) + 31) // 32)).astype(np.int32))
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, form)
    args = bt, ref.dev(ctx), ref.dev(prefix), ref.dev(cu), mask
    q = torch.randn((int(cu[-1]), hq, pool.head_dim), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    return cu, q, lambda q: pkv.pkv_tree_attn(pool, q, *args, 0.3)


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("hq,hkv", [(16, 2), (10, 2), (128, 1)])
def test_the_queries_beside_a_request_do_not_reach_it(form, dtype, hq, hkv):
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    pool = ref.random_pool(pkv.Pool(800, hkv, 128, **kw), 1)
    cu, q, call = batch(pool, 1, [3000, 2500, 2900, 2000], [5, 21, 3, 33], hq, form)
    want = None
    for k in range(4):
        x = q.clone()
        for r in (1, 3):                                   # requests 0 and 2 keep their queries
            x[cu[r]:cu[r + 1]] *= (0.0, 1.0, 30.0, -100.0)[k]
        o, lse = call(x)
        own = [t[cu[r]:cu[r + 1]].clone() for t in (o, lse) for r in (0, 2)]
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(pool) == 0
        want = want or own
        for a, b in zip(want, own):
            assert torch.equal(a, b), k
    pool.close()


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_calls_before_do_not_reach_it(form, dtype):
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    pool = ref.random_pool(pkv.Pool(900, 2, 128, **kw), 2)
    _, q, call = batch(pool, 2, [3000, 2500, 900, 3300], [25, 60, 110, 7], 10, form)    # tiles of 125 rows
    _, qp, poison = batch(pool, 3, [2000] * 5, [128, 64, 96, 32, 128], 8, form)          # of 128
    want = None
    for k in range(5):
        for _ in range(2):
            poison(qp * (0.0, 1.0, 40.0, -100.0, 1e4)[k])
        own = call(q)
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(pool) == 0
        want = want or own
        for a, b in zip(want, own):
            assert torch.equal(a, b), k
    pool.close()
