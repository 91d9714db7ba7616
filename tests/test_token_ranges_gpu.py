"""Token ranges that begin below 0 or end beyond the tokens: cut to the tokens there are, and flagged."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu

RANGES = [[-3, 2, 5], [0, 2, 9], [-1, 2, 6]]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class World:
    """Two requests of 2 and 3 tokens."""

    def __init__(self, width):
        self.pool = ref.random_pool(pkv.Pool(40, 2, 64), 1)
        self.bt = ref.dev(ref.tables(np.random.default_rng(1), [200, 300], 40, width))
        self.ctx, self.pos = ref.dev(np.array([200, 300], np.int32)), ref.dev(np.array([199, 40, 7, 299, 130], np.int32))
        self.q = torch.randn((5, 4, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        self.sum = pkv.BlockSummary(self.pool)

    def flags(self):
        torch.cuda.synchronize()
        return pkv.pkv_check_device_errors(self.pool)

    def both(self, call, cu, right=(0, 2, 5)):
        """call(cu) with the right ranges, then with `cu`: flagged, and the same results."""
        want = call(ref.dev(np.array(right, np.int32)))
        assert self.flags() == 0
        got = call(ref.dev(np.array(cu, np.int32)))
        assert self.flags() == pkv.PKV_DEVERR_POSITION
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cu", RANGES)
@pytest.mark.parametrize("width", [19, 600], ids=["one_kernel", "two_kernels"])
def test_bounds_selection_and_attention(cu, width):
    w = World(width)

    def bounds(cu):
        w.sum.codes.zero_()
        w.sum.exps.zero_()
        pkv.pkv_summarize(w.pool, w.sum, w.bt, cu, w.pos, w.ctx)
        return w.sum.codes.clone(), w.sum.exps.clone()

    w.both(bounds, cu)
    every = np.concatenate([np.arange(0, 200, 16), np.arange(0, 300, 16)]).astype(np.int32)
    pkv.pkv_summarize(w.pool, w.sum, w.bt, ref.dev(np.array([0, 13, 32], np.int32)), ref.dev(every), w.ctx)
    w.both(lambda cu: [pkv.pkv_select_blocks(w.pool, w.sum, w.q, w.pos, w.bt, cu, 5)], cu)
    sel = pkv.pkv_select_blocks(w.pool, w.sum, w.q, w.pos, w.bt, ref.dev(np.array([0, 2, 5], np.int32)), 5)
    w.both(lambda cu: pkv.pkv_sparse_attn(w.pool, w.q, w.pos, w.bt, cu, sel, 0.1), cu)


def test_bounds_of_prompts():
    """(16 tokens a warp)"""
    T = 64 * 160
    pool = ref.random_pool(pkv.Pool(T // 16, 1, 64), 1)
    bt, ctx = ref.dev(np.arange(T // 16, dtype=np.int32)[None]), ref.dev(np.array([T], np.int32))
    pos = ref.dev(np.arange(T, dtype=np.int32))
    got = []
    for cu, flag in (([0, T], 0), ([-1, T], pkv.PKV_DEVERR_POSITION), ([0, T + 1], pkv.PKV_DEVERR_POSITION)):
        s = pkv.BlockSummary(pool)
        pkv.pkv_summarize(pool, s, bt, ref.dev(np.array(cu, np.int32)), pos, ctx)
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(pool) == flag
        got.append(s)
    for s in got[1:]:
        assert torch.equal(s.codes, got[0].codes) and torch.equal(s.exps, got[0].exps)


@pytest.mark.parametrize("cu", [[0, 2, 9], [0, 2, 6]])
def test_masks_and_compaction(cu):
    w = World(19)
    parents = ref.dev(np.array([-1, 0, -1, 0, 1], np.int32))
    w.both(lambda cu: [pkv.pkv_tree_mask(w.pool, parents, cu, mask_words=1)], cu)
    src, dst = ref.dev(np.array([150, 160, 200, 220, 290], np.int32)), ref.dev(np.array([100, 30], np.int32))
    k0 = w.pool.k.clone()

    def move(cu):
        w.pool.k.copy_(k0)
        pkv.pkv_compact(w.pool, w.bt, cu, src, dst)
        return [w.pool.k.clone()]

    w.both(move, cu)


def test_a_range_that_begins_below_zero_leaves_its_mask_rows():
    """Node indexes count from the range's begin, so its rows are left alone; a compaction counts from its first kept."""
    w = World(19)
    out = torch.full((5, 1), 9, dtype=torch.int32, device="cuda")
    parents = ref.dev(np.array([-1, 0, -1, 0, 1], np.int32))
    pkv.pkv_tree_mask(w.pool, parents, ref.dev(np.array([-1, 2, 5], np.int32)), out=out)
    assert w.flags() & pkv.PKV_DEVERR_POSITION
    assert out[:, 0].tolist() == [9, 9, 1, 3, 7]
