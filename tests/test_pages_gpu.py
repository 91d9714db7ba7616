"""Page sharing, copying, allocating, freeing and compaction through the C ABI: whole numbers and bit copies, so every
result is compared for equality with a sequential restatement."""
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


def pages(n):
    return (n + 15) // 16


def fork_ref(tables, lens, caps, parents, new_caps, refs):
    """(new tables, new refs, copies [(src page, dst page, rows)]); None for a page that is not to be had."""
    refs = refs.astype(np.int64).copy()
    width = tables.shape[1]
    new = np.full((len(parents), width), -1, np.int64)
    kids = [[i for i, p in enumerate(parents) if p == r] for r in range(len(lens))]
    part_page = {}
    for r in range(len(lens)):
        full, part = lens[r] // 16, lens[r] % 16
        for j in range(pages(caps[r])):
            b = tables[r, j]
            if kids[r] and part and j == full:
                part_page[r] = b
            else:
                refs[b] -= 1
            if j < full:
                refs[b] += len(kids[r])
                for i in kids[r]:
                    new[i, j] = b
    owners = refs.copy()
    copies, late = [], []
    for r, b in part_page.items():
        movers = kids[r]
        if owners[b] == 1:
            new[movers[0], lens[r] // 16] = b
            movers = movers[1:]
        else:
            late.append(b)
        copies += [(i, r, b) for i in movers]
    free = [b for b in range(len(refs)) if owners[b] == 0][::-1]
    short = False
    for i, p in enumerate(parents):
        for j in range(pages(max(new_caps[i], lens[p] if p >= 0 else 0))):
            if new[i, j] < 0:
                if free:
                    new[i, j] = free.pop()
                    refs[new[i, j]] = 1
                else:
                    short = True
    for b in late:
        refs[b] -= 1
    moves = [(b, new[i, lens[r] // 16], lens[r] % 16) for i, r, b in copies if new[i, lens[r] // 16] >= 0]
    return new.astype(np.int32), refs.astype(np.int32), moves, short


class World:
    """Sequences over a pool, moved on by pkv_fork and by fork_ref side by side."""

    def __init__(self, seed, num_blocks, hkv=2, d=64, dtype="bf16", width=40):
        kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
        self.pool = ref.random_pool(pkv.Pool(num_blocks, hkv, d, **kw), seed)
        self.rng = np.random.default_rng(seed)
        self.sum = pkv.BlockSummary(self.pool)
        self.sum.codes.random_(-127, 127)
        self.sum.exps.random_(-20, 20)
        self.width = width
        self.tables = np.full((0, width), -1, np.int32)
        self.lens = self.caps = np.zeros(0, np.int32)
        self.refs = np.zeros(num_blocks, np.int32)

    def step(self, parents, new_caps, in_place=True, with_summary=False, expect_short=False):
        parents, new_caps = np.array(parents, np.int32), np.array(new_caps, np.int32)
        t = ref.dev
        k0, v0 = self.pool.k.clone(), self.pool.v.clone()
        c0, e0 = self.sum.codes.clone(), self.sum.exps.clone()
        refs = t(self.refs)
        out_refs = refs if in_place else torch.full_like(refs, -7)
        nt, nr = pkv.pkv_fork(self.pool, t(self.tables), t(self.lens), t(self.caps), t(parents), t(new_caps), refs,
                              out_refs=out_refs, summary=self.sum if with_summary else None)
        torch.cuda.synchronize()
        flags = pkv.pkv_check_device_errors(self.pool)
        want_t, want_r, moves, short = fork_ref(self.tables, self.lens, self.caps, parents, new_caps, self.refs)
        assert short == expect_short
        assert flags == (pkv.PKV_DEVERR_NO_PAGES if short else 0)
        assert np.array_equal(nr.cpu().numpy(), want_r)
        assert np.array_equal(nt.cpu().numpy(), want_t)
        for src, dst, rows in moves:
            k0[dst, :, :rows] = k0[src, :, :rows]
            v0[dst, :, :rows] = v0[src, :, :rows]
            if with_summary:
                c0[dst], e0[dst] = c0[src], e0[src]
        assert torch.equal(self.pool.k.view(torch.uint8), k0.view(torch.uint8))
        assert torch.equal(self.pool.v.view(torch.uint8), v0.view(torch.uint8))
        assert torch.equal(self.sum.codes, c0) and torch.equal(self.sum.exps, e0)
        if not in_place:
            assert np.array_equal(refs.cpu().numpy(), self.refs)
        inherited = np.array([self.lens[p] if p >= 0 else 0 for p in parents], np.int32)
        self.tables, self.refs = want_t, want_r
        self.caps = np.maximum(new_caps, inherited).astype(np.int32)
        self.lens = inherited
        return moves

    def grow(self, tokens):
        """The sequences take up tokens of their room."""
        self.lens = np.minimum(self.lens + np.asarray(tokens, np.int32), self.caps).astype(np.int32)


@pytest.mark.parametrize("dtype,d,hkv", [("bf16", 64, 2), ("bf16", 128, 3), ("fp8_e4m3", 64, 1), ("fp8_e4m3", 128, 5)])
@pytest.mark.parametrize("with_summary", [False, True])
def test_a_life_of_sequences(dtype, d, hkv, with_summary):
    w = World(d + hkv, 400, hkv, d, dtype)
    w.step([-1] * 5, [40, 16, 17, 1, 100], with_summary=with_summary)
    w.grow([33, 16, 17, 0, 64])
    for k in range(12):
        n = int(w.rng.integers(1, 9))
        parents = w.rng.integers(-1, len(w.lens), n)
        room = [int(w.lens[p] if p >= 0 else 0) + int(w.rng.integers(0, 40)) for p in parents]
        w.step(parents, room, in_place=k % 2 == 0, with_summary=with_summary)
        w.grow(w.rng.integers(0, 40, n))
    w.step([], [])                                        # all freed
    assert (w.refs == 0).all()


def test_no_rows_no_children_and_single_steps():
    w = World(1, 64)
    w.step([], [])
    w.step([-1], [1])
    w.grow([1])
    for _ in range(40):                                   # one sequence that grows token by token keeps its pages
        before = w.tables[0, :pages(w.lens[0])].copy()
        assert w.step([0], [w.lens[0] + 1]) == []
        assert np.array_equal(w.tables[0, :len(before)], before)
        w.grow([1])
    w.step([0, 0, 0], [w.lens[0]] * 3)                    # three children, no room wanted
    w.step([2, 2, -1], [0, 300, 5], in_place=False)


def test_pages_with_owners_elsewhere():
    w = World(2, 64)
    w.step([-1], [40])
    w.grow([40])
    w.refs[w.tables[0, :3]] += 1                          # someone keeps the prompt's pages, the partly filled one too
    assert len(w.step([0, 0], [41, 41])) == 2             # both children copy it
    assert len(w.step([0], [41])) == 0                    # the copy is its own
    # two rows that hold the same partly filled page, each continued once: both copy, the page becomes free
    w = World(3, 64)
    w.step([-1], [10])
    w.grow([10])
    w.tables = np.repeat(w.tables, 2, 0)
    w.lens, w.caps = np.repeat(w.lens, 2), np.repeat(w.caps, 2)
    w.refs[w.tables[0, 0]] = 2
    page = w.tables[0, 0]
    assert len(w.step([0, 1], [11, 11])) == 2
    assert w.refs[page] == 0


def test_too_few_pages():
    w = World(4, 9)
    w.step([-1, -1], [64, 60])
    w.grow([64, 60])
    w.step([0, 1, 1, 0], [70, 60, 60, 64], expect_short=True)
    w = World(5, 8)
    w.step([-1, -1], [64, 64])
    w.step([0, 0], [64, 64])                              # row 1's pages are given up and used again at once


def test_many_rows_and_pages():
    w = World(6, 5000, hkv=1, width=300)
    w.step([-1] * 40, [int(x) for x in w.rng.integers(1, 1500, 40)])
    w.grow(w.rng.integers(0, 1500, 40))
    parents = np.sort(w.rng.integers(0, 40, 2300))
    w.step(parents, [int(w.lens[p]) + 1 for p in parents])
    w.grow([1] * 2300)
    w.step(w.rng.integers(0, 2300, 1100), [0] * 1100)


def test_bad_arguments_on_the_device_are_flagged():
    w = World(7, 64)
    w.step([-1, -1], [40, 40])
    w.grow([20, 20])
    t = ref.dev

    def flags(tables=None, lens=None, caps=None, parents=(0, 1), new_caps=(30, 30)):
        refs = t(w.refs)
        nt, nr = pkv.pkv_fork(w.pool, t(w.tables if tables is None else tables), t(w.lens if lens is None else lens),
                              t(w.caps if caps is None else caps), t(np.array(parents, np.int32)),
                              t(np.array(new_caps, np.int32)), refs)
        torch.cuda.synchronize()
        return pkv.pkv_check_device_errors(w.pool), nt.cpu().numpy()

    bad = w.tables.copy()
    bad[0, 0], bad[1, 1] = -1, 64
    assert flags(tables=bad)[0] & pkv.PKV_DEVERR_BLOCK_ID
    f, nt = flags(parents=(0, 2))
    assert f == pkv.PKV_DEVERR_POSITION and (nt[1, :2] >= 0).all() and (nt[1, 2:] == -1).all()
    assert flags(parents=(-5, 0))[0] == pkv.PKV_DEVERR_POSITION
    assert flags(lens=np.array([41, 2], np.int32))[0] == pkv.PKV_DEVERR_POSITION
    assert flags(caps=np.array([-1, 40], np.int32))[0] == pkv.PKV_DEVERR_POSITION
    assert flags(caps=np.array([40, 2 ** 30], np.int32))[0] & pkv.PKV_DEVERR_POSITION


@pytest.mark.parametrize("dtype,d,hkv", [("bf16", 64, 2), ("fp8_e4m3", 128, 3), ("fp8_e4m3", 64, 1)])
def test_copy_blocks(dtype, d, hkv):
    w = World(8, 50, hkv, d, dtype)
    k0, v0, c0, e0 = (x.clone() for x in (w.pool.k, w.pool.v, w.sum.codes, w.sum.exps))
    src, dst = np.array([3, 3, 9, 49, 5], np.int32), np.array([0, 1, 20, 30, 5], np.int32)
    pkv.pkv_copy_blocks(w.pool, ref.dev(src), ref.dev(dst), summary=w.sum)
    for x in (k0, v0, c0, e0):
        x[torch.as_tensor(dst).long().cuda()] = x[torch.as_tensor(src).long().cuda()]
    for x, y in ((w.pool.k, k0), (w.pool.v, v0), (w.sum.codes, c0), (w.sum.exps, e0)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert pkv.pkv_check_device_errors(w.pool) == 0
    pkv.pkv_copy_blocks(w.pool, ref.dev(np.array([1, 50], np.int32)), ref.dev(np.array([-1, 2], np.int32)))
    assert pkv.pkv_check_device_errors(w.pool) == pkv.PKV_DEVERR_BLOCK_ID
    assert torch.equal(w.pool.k.view(torch.uint8), k0.view(torch.uint8))


@pytest.mark.parametrize("dtype,d,hkv", [("bf16", 64, 2), ("bf16", 128, 8), ("fp8_e4m3", 64, 1), ("fp8_e4m3", 128, 3)])
def test_compact(dtype, d, hkv):
    w = World(9, 120, hkv, d, dtype)
    rng = np.random.default_rng(9)
    base = np.array([0, 5, 16, 31, 100, 7], np.int32)
    drafts = [40, 64, 17, 1, 30, 20]
    bt = ref.tables(rng, [int(b) + n for b, n in zip(base, drafts)], 120)
    keep = [np.sort(rng.choice(n, k, replace=False)) for n, k in zip(drafts, [40, 20, 9, 1, 0, 13])]
    src = np.concatenate([b + x for b, x in zip(base, keep)]).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum([len(x) for x in keep])]).astype(np.int32)
    k0, v0 = w.pool.k.cpu(), w.pool.v.cpu()
    pkv.pkv_compact(w.pool, ref.dev(bt), ref.dev(cu), ref.dev(src), ref.dev(base))
    for x, y in ((k0, w.pool.k), (v0, w.pool.v)):
        old = x.clone()
        for r in range(6):
            for i in range(cu[r], cu[r + 1]):
                a, b = int(src[i]), int(base[r] + i - cu[r])
                x[int(bt[r, b // 16]), :, b % 16] = old[int(bt[r, a // 16]), :, a % 16]
        assert torch.equal(x.view(torch.uint8), y.cpu().view(torch.uint8))
    assert pkv.pkv_check_device_errors(w.pool) == 0


def test_compact_flags_what_it_cannot_move():
    w = World(10, 20)
    bt = ref.dev(np.arange(20, dtype=np.int32).reshape(1, 20))
    k0 = w.pool.k.clone()

    def move(src, dst, table=bt):
        src = np.array(src, np.int32)
        pkv.pkv_compact(w.pool, table, ref.dev(np.array([0, len(src)], np.int32)), ref.dev(src),
                        ref.dev(np.array([dst], np.int32)))
        return pkv.pkv_check_device_errors(w.pool)

    assert move([4, 5, 6], 4) == 0                          # nothing to move
    assert move([3], 4) == pkv.PKV_DEVERR_POSITION          # forwards
    assert move([320], 4) == pkv.PKV_DEVERR_POSITION        # outside the table
    assert move([40], 4, ref.dev(np.full((1, 20), 20, np.int32))) == pkv.PKV_DEVERR_BLOCK_ID
    assert torch.equal(w.pool.k, k0)
    assert move([9, 9], 4) == pkv.PKV_DEVERR_POSITION       # the second is not behind the first
    assert torch.equal(w.pool.k[0, :, 4], k0[0, :, 9]) and torch.equal(w.pool.k[0, :, 5:], k0[0, :, 5:])


def test_captured_step():
    w = World(11, 200)
    w.step([-1] * 4, [50, 60, 70, 80])
    w.grow([50, 55, 70, 70])
    t = ref.dev
    tables, lens, caps, refs = t(w.tables), t(w.lens), t(w.caps), t(w.refs)
    parents, room = t(np.array([0, 0, 2, 3], np.int32)), t(np.array([51, 51, 71, 71], np.int32))
    nt, nr = torch.empty_like(tables), torch.empty_like(refs)
    ws = torch.empty(pkv.pkv_fork_workspace_size(w.pool, 4, 4), dtype=torch.uint8, device="cuda")

    def call():
        pkv.pkv_fork(w.pool, tables, lens, caps, parents, room, refs, out_tables=nt, out_refs=nr, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for p in ([3, 3, 3, 3], [1, 0, 1, 2], [-1, 2, 2, 0]):
        parents.copy_(t(np.array(p, np.int32)))
        room.copy_(t(np.array([90, 91, 92, 93], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        want_t, want_r, _, _ = fork_ref(w.tables, w.lens, w.caps, p, [90, 91, 92, 93], w.refs)
        assert np.array_equal(nt.cpu().numpy(), want_t) and np.array_equal(nr.cpu().numpy(), want_r)


def test_drafting_step_end_to_end():
    """Append a tree of drafts, attend, keep one path, compact it: the kept tokens' outputs are those of the causal
    attention over the compacted cache, and two samples of the result are the result."""
    rng = np.random.default_rng(12)
    hq, hkv, d = 8, 2, 128
    prefix, n = np.array([45, 200, 3], np.int32), [12, 40, 7]
    ctx = (prefix + n).astype(np.int32)
    pool = ref.random_pool(pkv.Pool(64, hkv, d), 12)
    refs = torch.zeros(64, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    bt, _ = pkv.pkv_fork(pool, torch.zeros((0, 16), dtype=torch.int32, device="cuda"), none, none,
                         torch.full((3,), -1, dtype=torch.int32, device="cuda"), ref.dev(ctx), refs)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(cu[-1])
    parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, m)] for m in n]).astype(np.int32)
    slots = np.concatenate([np.arange(p, p + m) for p, m in zip(prefix, n)]).astype(np.int32)
    kn, vn, q = (torch.randn((T, h, d), device="cuda").to(torch.bfloat16) for h in (hkv, hkv, hq))
    pkv.pkv_append(pool, bt, ref.dev(cu), ref.dev(slots), kn, vn)
    mask = pkv.pkv_tree_mask(pool, ref.dev(parents), ref.dev(cu), max_nodes=max(n))
    o, lse = pkv.pkv_tree_attn(pool, q, bt, ref.dev(ctx), ref.dev(prefix), ref.dev(cu), mask, d ** -0.5)
    paths = []
    for r, m in enumerate(n):
        path, i = [], m - 1
        while i >= 0:
            path.insert(0, i)
            i = int(parents[cu[r] + i])
        paths.append(path)
    src = np.concatenate([prefix[r] + np.array(p) for r, p in enumerate(paths)]).astype(np.int32)
    cuk = np.concatenate([[0], np.cumsum([len(p) for p in paths])]).astype(np.int32)
    pkv.pkv_compact(pool, bt, ref.dev(cuk), ref.dev(src), ref.dev(prefix))
    lens = (prefix + np.diff(cuk)).astype(np.int32)
    two, _ = pkv.pkv_fork(pool, bt, ref.dev(lens), ref.dev(ctx), ref.dev(np.array([0, 0, 1, 1, 2, 2], np.int32)),
                          ref.dev(np.repeat(lens + 1, 2).astype(np.int32)), refs)
    kept = np.concatenate([cu[r] + np.array(p) for r, p in enumerate(paths)])
    pos = np.concatenate([np.arange(prefix[r], lens[r]) for r in range(3)]).astype(np.int32)
    K, V = ref.pool_values(pool, "k"), ref.pool_values(pool, "v")
    qk = q[torch.as_tensor(kept).cuda()].contiguous()
    for table in (bt, two[0::2].contiguous(), two[1::2].contiguous()):
        po, pl = pkv.pkv_paged_attn(pool, qk, ref.dev(pos), table, ref.dev(lens), ref.dev(cuk),
                                    pkv.HostMeta(cuk, lens, pos), d ** -0.5)
        torch.cuda.synchronize()
        t = table.cpu().numpy()
        for r in range(3):
            for g in range(hkv):
                k, _ = ref.gather(K, t[r], int(lens[r]), g)
                v, _ = ref.gather(V, t[r], int(lens[r]), g)
                a, b = cuk[r], cuk[r + 1]
                seen = np.repeat(np.arange(lens[r])[None] <= pos[a:b, None], hq // hkv, 0)
                rows = qk[a:b, g * 4:g * 4 + 4].float().double().cpu().numpy().reshape(-1, d)
                want, wl, to, tl = ref.softmax_rows(rows, k, v, seen, d ** -0.5, False)
                for oo, ll in ((po[a:b], pl[a:b]), (o[torch.as_tensor(kept[a:b]).cuda()], lse[torch.as_tensor(kept[a:b]).cuda()])):
                    ref.assert_close(oo[:, g * 4:g * 4 + 4].float().cpu().numpy().reshape(-1, d), want, to, "O")
                    ref.assert_close(ll[:, g * 4:g * 4 + 4].cpu().numpy().reshape(-1), wl, tl, "LSE")
    assert pkv.pkv_check_device_errors(pool) == 0


def test_refusals():
    w = World(13, 32)
    w.step([-1, -1], [20, 30])
    t = ref.dev
    tables, lens, caps, refs = t(w.tables), t(w.lens), t(w.caps), t(w.refs)
    one = t(np.array([0], np.int32))
    with pytest.raises(pkv.PkvError, match="overlap"):
        pkv.pkv_fork(w.pool, tables, lens, caps, t(np.array([0, 1], np.int32)), t(np.array([30, 30], np.int32)), refs,
                     out_tables=tables)
    with pytest.raises(pkv.PkvError, match="workspace"):
        pkv.pkv_fork(w.pool, tables, lens, caps, one, one, refs, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    for kw in (dict(lens=lens[:1]), dict(refs=refs[:5].contiguous()), dict(new_caps=t(np.zeros(2, np.int32)))):
        args = dict(tables=tables, lens=lens, caps=caps, parents=one, new_caps=one, refs=refs)
        args.update(kw)
        with pytest.raises(ValueError):
            pkv.pkv_fork(w.pool, **args)
    with pytest.raises(TypeError):
        pkv.pkv_fork(w.pool, tables.long(), lens, caps, one, one, refs)
    with pytest.raises(ValueError):
        pkv.pkv_copy_blocks(w.pool, one, t(np.zeros(2, np.int32)))
    with pytest.raises(ValueError):
        pkv.pkv_compact(w.pool, tables, one, one, one)
    lib = pkv.load_library()
    p = refs.data_ptr()
    assert lib.pkv_copy_blocks(w.pool.handle, p, p, 1, p, None, None) == pkv.PKV_EINVAL      # half a summary
    assert lib.pkv_copy_blocks(w.pool.handle, p, None, 1, None, None, None) == pkv.PKV_EINVAL
    assert lib.pkv_copy_blocks(w.pool.handle, p, p, -1, None, None, None) == pkv.PKV_EINVAL
    assert lib.pkv_compact(w.pool.handle, p, 1 << 28, 1, p, p, p, 1, None) == pkv.PKV_EINVAL
    assert np.array_equal(refs.cpu().numpy(), w.refs)


def test_nothing_to_do():
    w = World(14, 32)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    pkv.pkv_copy_blocks(w.pool, e, e)
    pkv.pkv_compact(w.pool, e.view(0, 3), torch.zeros(1, dtype=torch.int32, device="cuda"), e, e)
    assert pkv.pkv_check_device_errors(w.pool) == 0


def test_rows_around_the_limit_of_the_small_kernel():
    for rows, kids in ((1024, 1024), (1025, 3), (3, 1025), (1024, 1)):
        w = World(rows + kids, 6000, hkv=1, width=6)
        w.step([-1] * rows, w.rng.integers(1, 33, rows))
        w.grow(w.rng.integers(0, 33, rows))
        parents = w.rng.integers(-1, rows, kids)
        w.step(parents, w.rng.integers(1, 50, kids), in_place=False)


def test_pages_beyond_4_gb():
    nb = 600_000
    pool = pkv.Pool(nb, 2, 128)
    pool.k[-40:] = torch.randn((40, 2, 16, 128), device="cuda").to(torch.bfloat16)
    pool.v[-40:] = torch.randn((40, 2, 16, 128), device="cuda").to(torch.bfloat16)
    k, v = pool.k[-40:].clone(), pool.v[-40:].clone()
    refs = torch.ones(nb, dtype=torch.int32, device="cuda")
    refs[-30:] = 0                                           # the free pages are the last thirty
    base = nb - 40
    bt = np.array([[base, base + 1, -1]], np.int32)
    args = [bt, np.array([20], np.int32), np.array([32], np.int32), np.array([0, 0], np.int32), np.array([33, 33], np.int32)]
    want, want_refs, moves, short = fork_ref(*args, refs.cpu().numpy())
    assert want.tolist() == [[base, base + 1, base + 10], [base, base + 11, base + 12]] and not short
    assert moves == [(base + 1, base + 11, 4)]
    two, _ = pkv.pkv_fork(pool, *(ref.dev(x) for x in args), refs)
    assert np.array_equal(two.cpu().numpy(), want) and np.array_equal(refs.cpu().numpy(), want_refs)
    k[11, :, :4], v[11, :, :4] = k[1, :, :4], v[1, :, :4]
    pkv.pkv_copy_blocks(pool, ref.dev(np.array([base + 3], np.int32)), ref.dev(np.array([base + 20], np.int32)))
    k[20], v[20] = k[3], v[3]
    pkv.pkv_compact(pool, ref.dev(want[1:]), ref.dev(np.array([0, 2], np.int32)), ref.dev(np.array([19, 33], np.int32)),
                    ref.dev(np.array([16], np.int32)))
    for x in (k, v):
        a, b = x[11, :, 3].clone(), x[12, :, 1].clone()
        x[11, :, 0], x[11, :, 1] = a, b
    torch.cuda.synchronize()
    assert torch.equal(pool.k[-40:], k) and torch.equal(pool.v[-40:], v)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()


def test_a_closed_pool_is_refused():
    w = World(15, 32)
    t = ref.dev(np.zeros(1, np.int32))
    pkv.pkv_copy_blocks(w.pool, t, t)
    w.pool.close()
    never = pkv.Pool(4, 1, 64)
    never.close()
    for pool in (w.pool, never):
        with pytest.raises(pkv.PkvError, match="pool is NULL") as e:
            pkv.pkv_copy_blocks(pool, t, t)
        assert e.value.code == pkv.PKV_EINVAL


def test_arguments_of_other_types():
    w = World(16, 32)
    t = ref.dev(np.zeros(1, np.int32))
    with pytest.raises(AttributeError):
        pkv.pkv_copy_blocks(w.pool, t, t, stream=3)
    with pytest.raises(TypeError):
        pkv.pkv_copy_blocks(w.pool, t, None)
    with pytest.raises(TypeError):
        pkv.pkv_tree_mask(w.pool, t, ref.dev(np.array([0, 1], np.int32)), mask_words="two")
    with pytest.raises(ValueError):
        pkv.pkv_tree_mask(w.pool, t, ref.dev(np.array([0, 1], np.int32)), mask_words=1 << 40)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_tree_mask(w.pool, t, ref.dev(np.array([0, 1], np.int32)), mask_words=0)


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_calls_that_follow_one_another_see_what_the_last_one_wrote(dtype):
    """Moves, copies, forks, bounds, selections and attention without a wait between them, and with one: the same bits."""
    got = []
    for wait in (False, True):
        torch.manual_seed(17)                             # (the bounds that World makes up)
        w = World(17, 200, 8, 128, dtype, width=24)
        w.step([-1] * 6, [300] * 6)
        w.grow([300] * 6)
        rng = np.random.default_rng(18)
        bt, lens, caps, refs = ref.dev(w.tables), ref.dev(w.lens), ref.dev(w.caps), ref.dev(w.refs)
        tabs, counts = [bt, torch.zeros_like(bt)], [refs, torch.zeros_like(refs)]
        cu = ref.dev(np.arange(7).astype(np.int32))
        pos = ref.dev(np.full(6, 299, np.int32))
        same = ref.dev(np.arange(6).astype(np.int32))
        every = ref.dev(np.tile(np.arange(0, 300, 16), 6).astype(np.int32))
        every_cu = ref.dev((np.arange(7) * 19).astype(np.int32))
        q = torch.randn((6, 16, 128), generator=torch.Generator().manual_seed(19)).to(torch.bfloat16).cuda()
        mask = torch.full((6, 1), -1, dtype=torch.int32, device="cuda")
        prefix = ref.dev(np.full(6, 290, np.int32))
        moves = []
        for _ in range(20):
            src = np.concatenate([np.sort(rng.choice(np.arange(100, 300), 40, replace=False)) for _ in range(6)]).astype(np.int32)
            moves.append((ref.dev((np.arange(7) * 40).astype(np.int32)), ref.dev(src),
                          ref.dev(rng.integers(0, 100, 6).astype(np.int32))))
        torch.cuda.synchronize()
        outs = []

        def done():
            if wait:
                torch.cuda.synchronize()

        for k, (mcu, src, dst) in enumerate(moves):
            t, r = tabs[k % 2], counts[k % 2]
            pkv.pkv_compact(w.pool, t, mcu, src, dst)
            done()
            pkv.pkv_summarize(w.pool, w.sum, t, every_cu, every, lens)
            done()
            sel = pkv.pkv_select_blocks(w.pool, w.sum, q, pos, t, cu, 6)
            done()
            outs += [sel, *pkv.pkv_sparse_attn(w.pool, q, pos, t, cu, sel, 0.1)]
            done()
            outs += list(pkv.pkv_tree_attn(w.pool, q, t, lens, prefix, cu, mask, 0.1))
            done()
            pkv.pkv_fork(w.pool, t, lens, caps, same, lens, r, out_tables=tabs[(k + 1) % 2], out_refs=counts[(k + 1) % 2],
                         summary=w.sum)
            done()
            pkv.pkv_copy_blocks(w.pool, same + 190, same + 180, summary=w.sum)
            done()
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(w.pool) == 0
        got.append([x.view(torch.uint8).clone() for x in outs + [w.pool.k, w.pool.v, w.sum.codes, w.sum.exps] + tabs + counts])
    for a, b in zip(*got):
        assert torch.equal(a, b)
