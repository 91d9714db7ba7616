"""Forks of a cache of several pools (one a layer) under one set of tables: the same call on each, the counts changed by
the last."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv
from test_pages_gpu import fork_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_layers_get_the_same_tables_and_their_own_pages(dtype):
    from paged_kv_attention_25_gb300 import build
    build.build()
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    layers = [ref.random_pool(pkv.Pool(90, 2, 64, **kw), s) for s in range(4)]
    sums = [pkv.BlockSummary(p) for p in layers]
    for s in sums:
        s.codes.random_(-127, 128)
        s.exps.random_(-20, 20)
    rng = np.random.default_rng(3)
    tables = ref.tables(rng, [100, 60, 33, 5], 90, 12)
    lens = np.array([90, 60, 20, 5], np.int32)
    caps = np.array([100, 60, 33, 5], np.int32)
    parents, new_caps = np.array([0, 0, 2, 1, 1, 1, -1], np.int32), np.array([101, 91, 40, 61, 70, 60, 17], np.int32)
    refs = np.zeros(90, np.int32)
    refs[tables[tables >= 0]] = 1
    want, want_refs, moves, short = fork_ref(tables, lens, caps, parents, new_caps, refs)
    assert len(moves) == 3 and not short
    args = [ref.dev(x) for x in (tables, lens, caps, parents, new_caps)]
    counts = ref.dev(refs)
    spare = torch.empty_like(counts)
    new = torch.full((7, 12), 77, dtype=torch.int32, device="cuda")
    before = [[x.clone() for x in (p.k, p.v, s.codes, s.exps)] for p, s in zip(layers, sums)]
    for i, (p, s) in enumerate(zip(layers, sums)):
        pkv.pkv_fork(p, *args, counts, out_tables=new, out_refs=counts if i == 3 else spare, summary=s)
    torch.cuda.synchronize()
    assert np.array_equal(new.cpu().numpy(), want)
    assert np.array_equal(counts.cpu().numpy(), want_refs) and torch.equal(spare, counts)
    for p, s, old in zip(layers, sums, before):
        for src, dst, rows in moves:
            for x in old[:2]:
                x[dst, :, :rows] = x[src, :, :rows]
            for x in old[2:]:
                x[dst] = x[src]
        for x, y in zip((p.k, p.v, s.codes, s.exps), old):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert pkv.pkv_check_device_errors(p) == 0
        p.close()
