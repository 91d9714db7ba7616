"""Whose workspaces calls use: kept with the pool for torch's own streams, the call's own for a stream that may be
destroyed while its work runs."""
import ctypes

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


def test_streams_of_the_callers_own_leave_nothing_with_the_pool():
    cudart = ctypes.CDLL(next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line))
    pool = ref.random_pool(pkv.Pool(300, 2, 64), 1)
    bt, cu = ref.dev(np.arange(300, dtype=np.int32)[None]), ref.dev(np.array([0, 1], np.int32))
    pos = ref.dev(np.array([4790], np.int32))
    sel = ref.dev(np.tile(np.arange(300, dtype=np.int32), (1, 2, 1)))
    q = torch.randn((1, 8, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    o, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")

    def call():
        pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1, out=o, lse=lse)
        torch.cuda.current_stream().synchronize()
        return o.clone()

    size = pkv.pkv_sparse_attn_workspace_size(pool)
    held = torch.cuda.memory_allocated()
    want = call()
    assert torch.cuda.memory_allocated() - held >= size          # kept for the current stream
    del want
    want = call()
    with torch.cuda.stream(torch.cuda.Stream()):                 # and for another of torch's own
        held = torch.cuda.memory_allocated()
        got = call()
        assert torch.cuda.memory_allocated() - held >= size and torch.equal(got, want)
    for _ in range(3):
        raw = ctypes.c_void_p()
        assert cudart.cudaStreamCreateWithFlags(ctypes.byref(raw), 1) == 0
        with torch.cuda.stream(torch.cuda.ExternalStream(raw.value)):
            got = call()
            assert torch.equal(got, want)
            torch.cuda.current_stream().synchronize()
            del got
            held = torch.cuda.memory_allocated()
            call()
            assert torch.cuda.memory_allocated() <= held         # nothing is left there
        torch.cuda.synchronize()
        assert cudart.cudaStreamDestroy(raw) == 0
    pool.close()
