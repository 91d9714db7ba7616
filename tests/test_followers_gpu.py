"""Calls whose kernels may start before the kernels ahead of them end see what those wrote: bits with a wait after every
call, and without one."""
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


def both_ways(steps):
    """steps(done) -> outputs, run with done() = a wait and with done() = nothing; the outputs are equal."""
    got = []
    for done in (torch.cuda.synchronize, lambda: None):
        outs = steps(done)
        torch.cuda.synchronize()
        got.append([x.view(torch.uint8).clone() for x in outs])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("width", [40, 600], ids=["one_kernel", "two_kernels"])
@pytest.mark.parametrize("hkv", [3, 8])
def test_a_selection_behind_a_copy_of_pages_sees_the_copied_bounds(width, hkv):
    """Targets and sources are neighbouring pages, whose exponents share a sector; the tables hold the targets."""
    n, d = 30, 64
    nb = 4 * n
    pool = ref.random_pool(pkv.Pool(nb, hkv, d), 1)
    summary = pkv.BlockSummary(pool)
    gen = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(-127, 128, summary.codes.shape, generator=gen, device="cuda", dtype=torch.int8)
    exps = torch.randint(-20, 20, summary.exps.shape, generator=gen, device="cuda", dtype=torch.int8)
    bt = np.full((2, width), -1, np.int32)
    bt[0, :n] = np.arange(0, 2 * n, 2)                   # targets: the even pages
    bt[1, :n] = np.arange(2 * n, 4 * n, 2)
    bt, cu = ref.dev(bt), ref.dev(np.arange(3, dtype=np.int32))
    pos = ref.dev(np.full(2, n * 16 - 1, np.int32))
    q = torch.randn((2, 2 * hkv, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    pairs = []
    for k in range(20):
        perm = np.random.default_rng(k).permutation(2 * n)
        pairs.append((ref.dev((2 * perm + 1).astype(np.int32)), ref.dev((2 * np.arange(2 * n)).astype(np.int32))))

    def steps(done):
        summary.codes.copy_(codes)
        summary.exps.copy_(exps)
        torch.cuda.synchronize()
        outs = []
        for src, dst in pairs:
            pkv.pkv_copy_blocks(pool, src, dst, summary=summary)
            done()
            sel = pkv.pkv_select_blocks(pool, summary, q, pos, bt, cu, 7, sinks=1, recent=1)
            done()
            outs += [sel, *pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1)]
            done()
        return outs

    k0, v0 = pool.k.clone(), pool.v.clone()

    def from_the_start(done):
        pool.k.copy_(k0)
        pool.v.copy_(v0)
        return steps(done)

    both_ways(from_the_start)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
def test_an_attention_behind_a_mask_sees_its_rows(form):
    """One mask buffer, rewritten before every attention."""
    rng = np.random.default_rng(4)
    nodes = [40, 64, 9]
    prefix = np.array([500, 3, 1200], np.int32)
    ctx = (prefix + nodes).astype(np.int32)
    pool = ref.random_pool(pkv.Pool(140, 2, 128), 4)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, form)
    bt, cu = ref.dev(ref.tables(rng, ctx, 140)), ref.dev(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32))
    ctx, prefix = ref.dev(ctx), ref.dev(prefix)
    q = torch.randn((sum(nodes), 8, 128), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    parents = [ref.dev(np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(n)] for n in nodes])
                       .astype(np.int32)) for _ in range(20)]
    mask = torch.zeros((sum(nodes), 2), dtype=torch.int32, device="cuda")

    def steps(done):
        mask.zero_()
        outs = []
        for p in parents:
            pkv.pkv_tree_mask(pool, p, cu, out=mask)
            done()
            outs += list(pkv.pkv_tree_attn(pool, q, bt, ctx, prefix, cu, mask, 0.1))
            done()
        return outs

    both_ways(steps)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()


def test_an_attention_whose_queries_are_the_last_ones_outputs():
    pool = ref.random_pool(pkv.Pool(70, 2, 64), 5)
    bt = ref.dev(np.arange(60, dtype=np.int32).reshape(2, 30))
    cu, pos = ref.dev(np.arange(3, dtype=np.int32)), ref.dev(np.array([479, 300], np.int32))
    sel = ref.dev(np.tile(np.arange(30, dtype=np.int32), (2, 2, 1)))
    q0 = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    bufs = [torch.empty_like(q0), torch.empty_like(q0)]

    def steps(done):
        q, outs = q0, []
        for k in range(40):
            o, lse = pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 4.0, out=bufs[k % 2])
            done()
            outs.append(lse)
            q = o
        return outs + bufs

    both_ways(steps)
    pool.close()


def test_a_fork_behind_one_without_children_sees_its_counts():
    """Rows freed (no children) and started again, counts from one array to the other: no wait between the plans."""
    pool = pkv.Pool(300, 1, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    empty = torch.zeros((0, 20), dtype=torch.int32, device="cuda")
    start = ref.dev(np.full(8, -1, np.int32))
    room = ref.dev(np.full(8, 300, np.int32))

    def steps(done):
        a, b = torch.zeros(300, dtype=torch.int32, device="cuda"), torch.zeros(300, dtype=torch.int32, device="cuda")
        outs = []
        for _ in range(20):
            t, _ = pkv.pkv_fork(pool, empty, none, none, start, room, a, out_refs=b)
            done()
            pkv.pkv_fork(pool, t, room, room, none, none, b, out_refs=a)        # all freed
            done()
            t2, _ = pkv.pkv_fork(pool, empty, none, none, start, room, a, out_refs=b)
            done()
            outs += [t, t2, b.clone()]
            pkv.pkv_fork(pool, t2, room, room, none, none, b)
            done()
            a, b = b, a
        return outs + [a, b]

    both_ways(steps)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
def test_an_attention_behind_moved_rows_and_copied_pages_sees_them(form, dtype):
    """Compactions and page copies of the tables' own pages, each followed at once by the tree's and the lists' attention."""
    rng = np.random.default_rng(6)
    kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
    pool = ref.random_pool(pkv.Pool(200, 2, 128, **kw), 6)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, form)
    ctx = np.array([700, 90, 1100], np.int32)
    tables = ref.tables(rng, ctx, 200)
    bt, lens, cu = ref.dev(tables), ref.dev(ctx), ref.dev(np.array([0, 20, 40, 60], np.int32))
    pos = ref.dev(np.concatenate([np.arange(c - 20, c) for c in ctx]).astype(np.int32))
    prefix, mask = ref.dev(ctx - 20), torch.full((60, 1), 0xFFFFF, dtype=torch.int32, device="cuda")
    q = torch.randn((60, 16, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    sel = ref.dev(np.tile(np.arange(tables.shape[1], dtype=np.int32), (60, 2, 1)))
    used = np.unique(tables[tables >= 0])
    free = np.setdiff1d(np.arange(200), used)
    moves = []
    for _ in range(12):
        src = np.concatenate([np.sort(rng.choice(np.arange(40, c), 30, replace=False)) for c in ctx]).astype(np.int32)
        to = rng.permutation(used)[:40].astype(np.int32)
        moves.append((ref.dev(np.array([0, 30, 60, 90], np.int32)), ref.dev(src), ref.dev(rng.integers(0, 10, 3).astype(np.int32)),
                      ref.dev(rng.choice(free, 40).astype(np.int32)), ref.dev(to)))
    k0, v0 = pool.k.clone(), pool.v.clone()

    def steps(done):
        pool.k.copy_(k0)
        pool.v.copy_(v0)
        outs = []
        for mcu, src, dst, frm, to in moves:
            for change in (lambda: pkv.pkv_compact(pool, bt, mcu, src, dst), lambda: pkv.pkv_copy_blocks(pool, frm, to)):
                change()
                done()
                outs += list(pkv.pkv_tree_attn(pool, q, bt, lens, prefix, cu, mask, 0.1))
                done()
                change()
                done()
                outs += list(pkv.pkv_sparse_attn(pool, q, pos, bt, cu, sel, 0.1))
                done()
        return outs

    both_ways(steps)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()
