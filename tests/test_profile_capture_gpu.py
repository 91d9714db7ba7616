"""Kernel timing that is on while a call is captured: the captured launches are not timed, the eager ones are read."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_captured_launches_are_not_timed():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pool = ref.random_pool(pkv.Pool(40, 2, 64), 1)
    summary = pkv.BlockSummary(pool)
    bt, cu = ref.dev(np.arange(10, dtype=np.int32)[None]), ref.dev(np.array([0, 1], np.int32))
    pos, ctx = ref.dev(np.array([100], np.int32)), ref.dev(np.array([101], np.int32))

    def call():
        pkv.pkv_summarize(pool, summary, bt, cu, pos, ctx)

    call()
    torch.cuda.synchronize()
    pkv.pkv_profile_enable(pool, True)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    call()
    torch.cuda.synchronize()
    got = pkv.pkv_profile_read(pool, reset=True)["append"]
    assert got["launches"] == 2 and got["total_ms"] > 0
    call()
    torch.cuda.synchronize()
    assert pkv.pkv_profile_read(pool)["append"]["launches"] == 1
    pkv.pkv_profile_enable(pool, False)
    pool.close()
