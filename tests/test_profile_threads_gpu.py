"""Kernel timing while two threads make calls of one pool: every launch is counted."""
import threading

import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_launches_of_two_threads_are_counted():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pool = ref.random_pool(pkv.Pool(40, 2, 64), 1)
    summary = pkv.BlockSummary(pool)
    bt, cu = ref.dev(np.arange(10, dtype=np.int32)[None]), ref.dev(np.array([0, 1], np.int32))
    pos, ctx = ref.dev(np.array([100], np.int32)), ref.dev(np.array([101], np.int32))
    src, dst = ref.dev(np.array([20], np.int32)), ref.dev(np.array([30], np.int32))
    pkv.pkv_profile_enable(pool, True)
    torch.cuda.synchronize()
    calls = (lambda s: pkv.pkv_summarize(pool, summary, bt, cu, pos, ctx, stream=s),
             lambda s: pkv.pkv_copy_blocks(pool, src, dst, stream=s))

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(400):
            calls[i](s)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    got = 0
    for _ in range(20):                                     # read while the calls go on
        got += pkv.pkv_profile_read(pool, reset=True)["append"]["launches"]
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    got += pkv.pkv_profile_read(pool, reset=True)["append"]["launches"]
    assert got == 800
    pkv.pkv_profile_enable(pool, False)
    pool.close()
