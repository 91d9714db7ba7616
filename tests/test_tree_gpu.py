"""Tree attention through the C ABI against the formula in 64 bits (bounds: attn_ref)."""
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


@pytest.fixture(params=[1, 2], ids=["rows", "tiles"], autouse=True)
def form(request):
    """Every test runs with both kernels: on 16 rows, and on tiles of 128."""
    Case.form = request.param


class Case:
    """A batch of drafted trees over a pool of random values."""

    def __init__(self, seed, reqs, hq, hkv, d, dtype="bf16", words=None, extra_tokens=0, kind="tree", scales=(0.02, 0.5)):
        """reqs: (prefix, drafts, query tokens or None for all drafts)."""
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.g = hq, hkv, d, hq // hkv
        self.prefix = np.array([r[0] for r in reqs], np.int32)
        drafts = [r[1] for r in reqs]
        self.ctx = np.array([p + n for p, n in zip(self.prefix, drafts)], np.int32)
        nq = [r[1] if len(r) < 3 else r[2] for r in reqs]
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_tokens
        nblk = sum((int(c) + 15) // 16 for c in self.ctx) + 5
        kw = dict(dtype=dtype, k_scale=scales[0], v_scale=scales[1]) if dtype != "bf16" else {}
        self.pool = ref.random_pool(pkv.Pool(nblk, hkv, d, **kw), seed)
        pkv.pkv_debug_set(self.pool, pkv.PKV_DEBUG_TREE_FORM, self.form)
        self.bt = ref.tables(rng, self.ctx, nblk)
        self.words = max(1, (max(drafts + [1]) + 31) // 32) if words is None else words
        self.bits = np.zeros((self.T, self.words * 32), bool)
        for r, n in enumerate(drafts):
            for i in range(nq[r]):
                node = n - nq[r] + i                     # the query tokens are the last nodes
                if kind == "tree":
                    anc = {node}
                    while node > 0 and rng.random() < 0.9:
                        node = int(rng.integers(max(0, node - 6), node))
                        anc.add(node)
                    for j in anc:
                        self.bits[self.cu[r] + i, j] = True
                elif kind == "random":
                    self.bits[self.cu[r] + i] = rng.random(self.words * 32) < 0.5
        self.q = torch.randn((self.T, hq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        self.scale = d ** -0.5

    def mask(self):
        w = self.bits.reshape(self.T, self.words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)
        return ref.dev(w.sum(-1).astype(np.uint32).view(np.int32))

    def run(self, **kw):
        return pkv.pkv_tree_attn(self.pool, self.q, ref.dev(self.bt), ref.dev(self.ctx), ref.dev(self.prefix),
                                 ref.dev(self.cu), self.mask(), self.scale, **kw)

    def check(self, o, lse):
        torch.cuda.synchronize()
        K, V = ref.pool_values(self.pool, "k"), ref.pool_values(self.pool, "v")
        q = self.q.float().double().cpu().numpy()
        o = o.float().cpu().numpy()
        lse = lse.cpu().numpy()
        for r in range(len(self.ctx)):
            a, b, ctx, pre = self.cu[r], self.cu[r + 1], int(self.ctx[r]), int(self.prefix[r])
            if a == b:
                continue
            slot = np.arange(ctx)
            bit = np.clip(slot - pre, 0, self.words * 32 - 1)
            seen = (slot < pre) | (self.bits[a:b][:, bit] & (slot - pre < self.words * 32))
            for g in range(self.hkv):
                k, good = ref.gather(K, self.bt[r], ctx, g)
                v, _ = ref.gather(V, self.bt[r], ctx, g)
                rows = q[a:b, g * self.g:(g + 1) * self.g].reshape(-1, self.d)
                want, wl, to, tl = ref.softmax_rows(rows, k, v, np.repeat(seen & good, self.g, 0), self.scale,
                                                    self.pool.dtype != "bf16")
                got = o[a:b, g * self.g:(g + 1) * self.g].reshape(-1, self.d)
                ref.assert_close(got, want, to, f"O of request {r}, head {g}")
                ref.assert_close(lse[a:b, g * self.g:(g + 1) * self.g].reshape(-1), wl, tl, f"LSE of request {r}, head {g}")

    def run_check(self, **kw):
        o, lse = self.run(**kw)
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(self.pool) == 0
        self.check(o, lse)


SMALL = [(0, 1), (0, 17), (1, 1), (15, 1), (16, 5), (17, 40), (0, 0), (127, 3), (128, 33), (250, 7), (5, 64), (400, 1)]


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 2, 64), (4, 4, 128), (8, 1, 128), (15, 3, 128), (32, 2, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_small_trees(hq, hkv, d, dtype):
    Case(hq * 100 + d, SMALL, hq, hkv, d, dtype).run_check()


@pytest.mark.parametrize("reqs", [[(0, 1)], [(1, 1)], [(0, 0), (33, 2)], [(16, 16)], [(3000, 1)], [(5000, 64), (3, 1)]])
def test_lone_requests(reqs):
    Case(3, reqs, 8, 2, 128).run_check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_large_group_and_long_context(dtype):
    Case(5, [(9000, 20), (40, 3)], 128, 1, 128, dtype).run_check()
    Case(6, [(2100, 64), (700, 31), (129, 64)], 64, 8, 128, dtype).run_check()


def test_many_requests():
    rng = np.random.default_rng(7)
    Case(7, [(int(rng.integers(0, 60)), int(rng.integers(0, 5))) for _ in range(700)], 4, 2, 64).run_check()


def test_masks_that_leave_rows_empty():
    Case(8, [(0, 9), (20, 9), (0, 40)], 8, 2, 64, kind="none").run_check()


def test_any_mask_and_words_beyond_and_short_of_the_tree():
    Case(9, [(20, 70), (0, 33), (7, 5)], 8, 2, 64, kind="random").run_check()
    Case(10, [(20, 70), (0, 33), (7, 5)], 8, 2, 64, kind="random", words=6).run_check()
    Case(11, [(20, 70), (0, 33), (7, 5)], 8, 2, 64, kind="random", words=1).run_check()
    Case(12, [(600, 500), (3, 300)], 8, 2, 64, kind="random").run_check()


def test_query_tokens_that_are_the_newest_nodes_only():
    Case(13, [(50, 30, 4), (0, 64, 1), (128, 10, 0), (77, 40, 17)], 8, 2, 128, kind="random").run_check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_values_in_unseen_slots_do_not_matter(dtype):
    """NaN behind the context, in blocks of no request, and (K, and V with infinities) in slots that rows do not see."""
    c = Case(14, [(37, 11), (0, 6), (160, 64)], 8, 2, 128, dtype)
    nan = 0x7F if dtype != "bf16" else float("nan")
    for x in (c.pool.k, c.pool.v):
        used = np.unique(c.bt[c.bt >= 0])
        free = np.setdiff1d(np.arange(c.pool.num_blocks), used)
        x[torch.as_tensor(free).cuda()] = nan
        for r, ctx in enumerate(c.ctx):
            if ctx % 16:
                x[int(c.bt[r, ctx // 16]), :, ctx % 16:] = nan
        for r, node in ((0, 3), (2, 20)):                  # a node that only some rows see
            slot = int(c.prefix[r]) + node
            x[int(c.bt[r, slot // 16]), :, slot % 16, 5:9] = nan
        if dtype == "bf16":
            slot = int(c.prefix[2]) + 30
            c.pool.v[int(c.bt[2, slot // 16]), :, slot % 16, 70] = float("inf")
            c.pool.v[int(c.bt[2, slot // 16]), :, slot % 16, 71] = float("-inf")
    o, lse = c.run()
    c.check(o, lse)
    # Rows that do not see the poisoned nodes are finite.
    fine = ~(c.bits[c.cu[2]:c.cu[3], 20] | c.bits[c.cu[2]:c.cu[3], 30])
    assert torch.isfinite(o[c.cu[2]:c.cu[3]][torch.as_tensor(fine).cuda()].float()).all()


def test_rows_behind_the_last_request_are_left_alone():
    c = Case(15, [(40, 5), (10, 3)], 8, 2, 64, extra_tokens=9)
    out = torch.full_like(c.q, 7.0)
    lse = torch.full((c.T, 8), 3.0, device="cuda")
    c.run(out=out, lse=lse)
    c.check(out, lse)
    assert (out[c.cu[-1]:] == 7.0).all() and (lse[c.cu[-1]:] == 3.0).all()


def test_bad_ids_and_lengths_are_flagged_and_skipped():
    c = Case(16, [(100, 5), (64, 12), (30, 30)], 8, 2, 64)
    c.bt[0, 2] = -1
    c.bt[1, 4] = c.pool.num_blocks
    o, lse = c.run()
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_BLOCK_ID
    c.check(o, lse)
    c = Case(17, [(100, 5), (64, 12)], 8, 2, 64)
    c.ctx[1] = c.bt.shape[1] * 16 + 1
    c.run()
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_POSITION


def test_runs_are_repeatable_and_lse_is_optional():
    c = Case(18, [(1500, 40), (3000, 64), (10, 1)], 64, 8, 128)
    a, la = c.run()
    b, none = c.run(want_lse=False)
    assert none is None
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_other_stream_and_own_workspace():
    c = Case(19, [(700, 33), (90, 12)], 8, 2, 128)
    ws = torch.empty(pkv.pkv_tree_attn_workspace_size(c.pool, 8, c.bt.shape[1], 2, c.T), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = c.run(stream=s, workspace=ws)
    s.synchronize()
    c.check(o, lse)


def test_captured_call_follows_lengths_tables_and_masks():
    c = Case(20, [(300, 20), (40, 20), (0, 20)], 8, 2, 128)
    bt, ctx, pre, cu, mask = (
        ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.prefix), ref.dev(c.cu), c.mask())
    out, lse = torch.zeros_like(c.q), torch.zeros((c.T, 8), device="cuda")
    ws = torch.empty(pkv.pkv_tree_attn_workspace_size(c.pool, 8, c.bt.shape[1], 3, c.T), dtype=torch.uint8, device="cuda")

    def call():
        pkv.pkv_tree_attn(c.pool, c.q, bt, ctx, pre, cu, mask, c.scale, out=out, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        # other lengths and query counts over the same tables
        c.prefix = np.array([300 - 50 * k, 40 - 10 * k, 0], np.int32)
        c.ctx = c.prefix + np.array([20, 12 + k, 9], np.int32)
        c.cu = np.array([0, 20 - k, 30, 39 + k], np.int32)
        c.bits = np.random.default_rng(k).random(c.bits.shape) < 0.5
        for t, x in ((ctx, c.ctx), (pre, c.prefix), (cu, c.cu)):
            t.copy_(ref.dev(x))
        mask.copy_(c.mask())
        c.q.copy_(torch.randn(c.q.shape, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
    assert pkv.pkv_check_device_errors(c.pool) == 0


def test_trees_of_many_tiles():
    """1 to 9 tiles of 128 rows, ragged last ones, over contexts that are cut between workers."""
    Case(22, [(200, 9), (1000, 130), (77, 65), (300, 40), (2000, 33), (64, 17), (5, 50), (129, 1)], 64, 8, 64).run_check()
    Case(23, [(3000, 100), (10, 51), (500, 26)], 15, 3, 128).run_check()
    Case(24, [(1500, 9), (20, 4), (130, 1)], 128, 1, 128).run_check()
    Case(25, [(700, 290)], 16, 4, 128, "fp8_e4m3").run_check()


def test_large_logits():
    c = Case(21, [(900, 30)], 8, 2, 64)
    c.scale = 4.0
    c.run_check()


@pytest.mark.parametrize("words", [1, 2, 40])
def test_mask_from_parents(words):
    rng = np.random.default_rng(words)
    counts = [0, 1, 5, 32, min(64, words * 32), 0, 17 if words == 1 else 33]
    counts = [min(n, words * 32) for n in counts]
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(cu[-1]) + 3
    parents = np.full(T, -1, np.int32)
    want = np.zeros((T, words * 32), bool)
    for r, n in enumerate(counts):
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -1
            parents[cu[r] + i] = p
            if p >= 0:
                want[cu[r] + i] = want[cu[r] + p]
            want[cu[r] + i, i] = True
    pool = pkv.Pool(4, 1, 64)
    out = torch.full((T, words), 99, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_mask(pool, ref.dev(parents), ref.dev(cu), out=out)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(pool) == 0
    got = out.cpu().numpy().view(np.uint32)
    bits = ((got[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool).reshape(T, -1)
    assert np.array_equal(bits[:cu[-1]], want[:cu[-1]])
    assert (got[cu[-1]:] == 99).all()
    parents[cu[2] + 2] = 2                      # its own parent
    pkv.pkv_tree_mask(pool, ref.dev(parents), ref.dev(cu), out=out)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(pool) == pkv.PKV_DEVERR_POSITION


def test_wait_that_runs_out_is_reported_and_the_pool_recovers():
    if Case.form == 1:
        return                                            # the rows form waits on no barrier
    for dtype in ("bf16", "fp8_e4m3"):
        c = Case(30, [(3000, 20), (500, 33), (40, 3)], 8, 2, 128, dtype)
        pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WAIT_LIMIT_NS, 2_000_000)
        pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WITHHOLD_COPY, Case.form)
        c.run()
        assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_TIMEOUT
        pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WITHHOLD_COPY, 0)
        pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WAIT_LIMIT_NS, 1_000_000_000)
        c.run_check()


def test_refusals():
    c = Case(31, [(20, 5)], 8, 2, 64)
    bt, ctx, pre, cu, mask = ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.prefix), ref.dev(c.cu), c.mask()

    def call(q=c.q, bt=bt, ctx=ctx, pre=pre, cu=cu, mask=mask, scale=0.1, **kw):
        return pkv.pkv_tree_attn(c.pool, q, bt, ctx, pre, cu, mask, scale, **kw)

    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(pkv.PkvError) as e:
            call(scale=scale)
        assert e.value.code == pkv.PKV_EINVAL
    odd = torch.zeros(c.q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(c.q.shape)
    for kw in (dict(q=odd), dict(out=odd)):
        with pytest.raises(pkv.PkvError, match="aligned"):
            call(**kw)
    with pytest.raises(pkv.PkvError, match="workspace"):
        call(workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pkv.PkvError, match="aligned"):
        n = pkv.pkv_tree_attn_workspace_size(c.pool, 8, c.bt.shape[1], 1, c.T)
        call(workspace=torch.empty(n + 512, dtype=torch.uint8, device="cuda")[8:])
    q3 = torch.zeros((c.T, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError, match="multiple"):
        call(q=q3)
    with pytest.raises(pkv.PkvError) as e:
        call(q=torch.zeros((c.T, 2 * 129, 64), dtype=torch.bfloat16, device="cuda"))
    assert e.value.code == pkv.PKV_EUNSUPPORTED
    with pytest.raises(TypeError):
        call(q=c.q.float())
    with pytest.raises(TypeError):
        call(q=torch.zeros((c.T, 64, 8), dtype=torch.bfloat16, device="cuda").transpose(1, 2))
    with pytest.raises(TypeError):
        call(mask=mask.long())
    for kw in (dict(ctx=torch.cat([ctx, ctx])), dict(pre=pre[:0]), dict(mask=mask[:-1].contiguous()),
               dict(bt=torch.cat([bt, bt])), dict(lse=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)


def test_no_tokens_is_nothing_to_do():
    c = Case(32, [(20, 5)], 8, 2, 64)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.q[:0]
    o, lse = pkv.pkv_tree_attn(c.pool, q, e.view(0, 3), e, e, zero, e.view(0, 1), 0.1)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    # requests without query tokens beside a padded batch: nothing is written
    out = torch.full_like(c.q, 7.0)
    pkv.pkv_tree_attn(c.pool, c.q, ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.prefix), torch.cat([zero, zero]), c.mask(),
                      0.1, out=out)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and pkv.pkv_check_device_errors(c.pool) == 0


def test_output_at_an_odd_multiple_of_16_bytes():
    c = Case(33, [(600, 40), (33, 7)], 8, 2, 128)
    out = torch.zeros(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(c.q.shape)
    o, lse = c.run(out=out)
    c.check(o, lse)


def test_two_threads_and_two_streams_at_once():
    """Calls of one pool from two threads: on one stream (they share the pool's workspace) and on two."""
    import threading
    cases = [Case(34, [(3000, 20), (100, 9)], 8, 2, 128), Case(35, [(2500, 33), (700, 5)], 8, 2, 128)]
    cases[1].pool.close()
    cases[1].pool = cases[0].pool
    nb = cases[0].pool.num_blocks
    rng = np.random.default_rng(1)
    for c in cases:                       # tables that may share blocks: the pool is only read
        c.bt = np.where(c.bt >= 0, rng.integers(0, nb, c.bt.shape), -1).astype(np.int32)
    for streams in ((None, None), (torch.cuda.Stream(), torch.cuda.Stream())):
        got = [None, None]
        args = [(c.pool, c.q, ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.prefix), ref.dev(c.cu), c.mask(), c.scale) for c in cases]
        torch.cuda.synchronize()

        def work(i):
            for _ in range(30):
                got[i] = pkv.pkv_tree_attn(*args[i], stream=streams[i])

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for c, (o, lse) in zip(cases, got):
            c.check(o, lse)


def test_graph_with_its_own_workspace_beside_eager_calls():
    c = Case(36, [(900, 20), (40, 20)], 8, 2, 64)
    args = (c.pool, c.q, ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.prefix), ref.dev(c.cu), c.mask(), c.scale)
    pkv.pkv_tree_attn(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = pkv.pkv_tree_attn(*args)
    s = torch.cuda.Stream()
    for _ in range(5):                    # the replay on one stream, eager calls on another, at the same time
        with torch.cuda.stream(s):
            graph.replay()
        o2, lse2 = pkv.pkv_tree_attn(*args)
    torch.cuda.synchronize()
    c.check(o, lse)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_blocks_beyond_4_gb():
    """Offsets above 2^32 bytes: a pool of 4.9 GB of K, its requests in the last blocks."""
    if Case.form == 1:
        c = Case(37, [(700, 20), (40, 7)], 8, 2, 128)
    else:
        c = Case(37, [(700, 40), (40, 7)], 8, 2, 128)
    nb, small = 600_000, c.pool
    pool = pkv.Pool(nb, 2, 128)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, Case.form)
    pool.k[nb - small.num_blocks:] = small.k
    pool.v[nb - small.num_blocks:] = small.v
    o, lse = pkv.pkv_tree_attn(pool, c.q, ref.dev(np.where(c.bt >= 0, c.bt + nb - small.num_blocks, -1).astype(np.int32)),
                               ref.dev(c.ctx), ref.dev(c.prefix), ref.dev(c.cu), c.mask(), c.scale)
    c.check(o, lse)
    assert pkv.pkv_check_device_errors(pool) == 0
    pool.close()


def test_query_tokens_over_an_empty_cache():
    c = Case(38, [(0, 4), (30, 6), (0, 40)], 8, 2, 128)
    c.ctx[:] = [0, 36, 0]
    c.prefix[:] = [0, 30, 0]
    o, lse = c.run()
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) == 0
    for a, b in ((0, 4), (10, 50)):
        assert (o[a:b] == 0).all() and (lse[a:b] == float("-inf")).all()
    c.check(o, lse)


def test_prefixes_out_of_range_are_flagged():
    for prefix in (-1, 200):
        c = Case(39, [(20, 5), (40, 3)], 8, 2, 64)
        c.prefix[0] = prefix
        o, lse = c.run()
        torch.cuda.synchronize()
        assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_POSITION
        c.prefix[0] = min(max(prefix, 0), c.ctx[0])          # cut to its range
        c.check(o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("reqs", [[(3000, 90), (1700, 200)], [(600, 20)] * 30, [(1000, 150)] * 4], ids=["long", "many", "several"])
def test_infinite_values_that_some_rows_see_in_groups_of_every_sharing(dtype, reqs):
    """V of NaN or infinities in tree slots, in groups that are whole, cut between CTAs, or shared out over warps."""
    c = Case(40, reqs, 16, 8, 128, dtype, kind="random")
    rng = np.random.default_rng(41)
    for r in range(len(reqs)):
        for slot in rng.integers(c.prefix[r], c.ctx[r], 3):
            row = c.pool.v[int(c.bt[r, slot // 16]), int(rng.integers(0, 8)), int(slot) % 16]
            if dtype == "bf16":
                row[int(rng.integers(0, 128))] = float(rng.choice([np.inf, -np.inf, np.nan]))
            else:
                row[int(rng.integers(0, 128))] = 0x7F
    c.run_check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_whole_groups_of_six_and_twelve_warps(dtype, d):
    rng = np.random.default_rng(42)
    reqs = [(int(rng.integers(0, 480)), int(rng.integers(0, 9))) for _ in range(25)]
    Case(43, reqs, 8, 8, d, dtype).run_check()               # at most 248 groups of 31 blocks
    Case(44, reqs[:5] + [(1000, 12)], 8, 8, d, dtype, kind="random").run_check()
    Case(45, [(1800, 9), (1700, 16), (900, 1)], 16, 16, d, dtype).run_check()   # 48 of 114
