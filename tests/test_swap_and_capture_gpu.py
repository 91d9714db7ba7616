"""A pending ahead-of-time swap-in and captured calls: a capture is refused without ending it, and after
pkv_swap_in_finish the replay reads the blocks."""
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


def test_a_swap_in_is_finished_before_a_capture_and_before_a_replay():
    pool = ref.random_pool(pkv.Pool(20, 2, 64), 1)
    t = ref.dev
    bt, cu = t(np.arange(10, dtype=np.int32)[None]), t(np.array([0, 1], np.int32))
    ctx, prefix, pos = t(np.array([150], np.int32)), t(np.array([149], np.int32)), t(np.array([149], np.int32))
    mask = t(np.array([[1]], np.int32))
    sel = t(np.tile(np.arange(10, dtype=np.int32), (1, 2, 1)))
    q = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    summary = pkv.BlockSummary(pool)
    one = t(np.array([0], np.int32))
    refs = torch.ones(20, dtype=torch.int32, device="cuda")
    calls = [lambda: pkv.pkv_tree_attn(pool, q, bt, ctx, prefix, cu, mask, 0.1),
             lambda: pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1),
             lambda: pkv.pkv_summarize(pool, summary, bt, cu, pos, ctx),
             lambda: pkv.pkv_fork(pool, bt, ctx, ctx, one, ctx, refs),
             lambda: pkv.pkv_copy_blocks(pool, one + 15, one + 16),
             lambda: pkv.pkv_compact(pool, bt, cu, one + 7, one + 3)]
    for call in calls:                                     # (kernels loaded before the capture)
        call()
    torch.cuda.synchronize()
    host = torch.randn((3, 2, 2, 16, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).pin_memory()
    copy = torch.cuda.Stream()
    ids = np.array([2, 5, 9], np.int32)

    pkv.pkv_swap_in_ahead(pool, ids, host, copy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            with pytest.raises(pkv.PkvError, match="swap-in is pending") as e:
                call()
            assert e.value.code == pkv.PKV_EINVAL
        keep = q + 1                                       # the capture goes on
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(keep, q + 1)
    pkv.pkv_swap_in_finish(pool)
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
        o, lse = calls[0]()
    pkv.pkv_swap_in_ahead(pool, ids, host.flip(0).contiguous().pin_memory(), copy)
    pkv.pkv_swap_in_finish(pool)
    graph.replay()
    want, wl = calls[0]()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert torch.equal(pool.k[torch.as_tensor(ids).long().cuda()].cpu(), host.flip(0)[:, 0])
    pool.close()


def test_a_swap_in_that_is_started_and_landed_in_one_capture():
    pool = ref.random_pool(pkv.Pool(20, 2, 64), 3)
    bt, cu = ref.dev(np.arange(10, dtype=np.int32)[None]), ref.dev(np.array([0, 1], np.int32))
    pos = ref.dev(np.array([149], np.int32))
    sel = ref.dev(np.tile(np.arange(10, dtype=np.int32), (1, 2, 1)))
    q = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1)
    host = torch.randn((3, 2, 2, 16, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).pin_memory()
    ids = np.array([2, 5, 9], np.int32)
    copy = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):       # (the staging buffer is allocated here)
        pkv.pkv_swap_in_ahead(pool, ids, host, copy)
        o, lse = pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool.k[torch.as_tensor(ids).long().cuda()].cpu(), host[:, 0])
    want, wl = pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    pool.close()
