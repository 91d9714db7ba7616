"""Bounds, block selection and attention over selected blocks, through the C ABI, against their definitions.

Bounds and selection are whole numbers: equal, not close.  The attention's bounds: attn_ref.
"""
import math

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


def raw_k(pool):
    """K in the units of the bounds (codes' values without the scale)."""
    x = pool.k.cpu()
    return (x.view(torch.float8_e4m3fn).float() if x.dtype == torch.uint8 else x.float()).double().numpy()


def unit(amax, most, least=-126):
    """The smallest exponent e >= least with amax <= most * 2^e, by trial."""
    if amax == 0:
        return least
    e = max(least, math.frexp(amax / most)[1] + 1)
    while e > least and amax <= math.ldexp(most, e - 1):
        e -= 1
    return e


def bounds_of(keys):
    """keys [n, D] float64 -> codes [2, D], exponent."""
    most = float(torch.finfo(torch.bfloat16).max)
    with np.errstate(invalid="ignore"):
        hi = np.fmax.reduce(np.clip(keys, -most, most), 0)
        lo = np.fmin.reduce(np.clip(keys, -most, most), 0)
    hi, lo = np.where(np.isnan(hi), 0.0, hi), np.where(np.isnan(lo), 0.0, lo)
    e = unit(max(np.abs(hi).max(), np.abs(lo).max()), 127.0)
    return np.stack([np.ceil(np.ldexp(hi, -e)), np.floor(np.ldexp(lo, -e))]).astype(np.int64), e


def scores(q, codes, exps):
    """q [G, D] float64, codes [n, 2, D] int64, exps [n] -> fp32 scores as float64."""
    G = q.shape[0]
    most = 32767 // G
    q = np.where(np.isfinite(q), q, 0.0)
    amax = np.abs(q).max()
    i = np.zeros(q.shape, np.int64) if amax < 2.0 ** -100 else np.rint(np.ldexp(q, -unit(amax, most, -300))).astype(np.int64)
    P, N = np.maximum(i, 0).sum(0), np.minimum(i, 0).sum(0)
    whole = codes[:, 0] @ P + codes[:, 1] @ N
    assert np.abs(whole).max(initial=0) < 2 ** 30
    with np.errstate(over="ignore"):        # the product in fp32: infinite above its range, subnormal below
        return np.ldexp(whole.astype(np.float32).astype(np.float64), exps).astype(np.float32).astype(np.float64)


def choose(score, valid, k, sinks, recent):
    n = len(score)
    j = np.arange(n)
    forced = (j < sinks) | (j >= n - recent)
    order = sorted(range(n), key=lambda b: (not valid[b], not forced[b], 0.0 if forced[b] else -score[b], b))[:k]
    sel = sorted(b for b in order if valid[b])
    return np.array(sel + [-1] * (k - len(sel)), np.int32)


class Case:
    def __init__(self, seed, reqs, hq, hkv, d, dtype="bf16", extra_tokens=0, width=None):
        """reqs: (context, query positions)."""
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.g = hq, hkv, d, hq // hkv
        self.ctx = np.array([r[0] for r in reqs], np.int32)
        self.pos = np.concatenate([np.asarray(r[1], np.int32) for r in reqs] + [np.zeros(extra_tokens, np.int32)]).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum([len(r[1]) for r in reqs])]).astype(np.int32)
        self.T = len(self.pos)
        nblk = sum((int(c) + 15) // 16 for c in self.ctx) + 4
        kw = dict(dtype=dtype, k_scale=0.02, v_scale=0.5) if dtype != "bf16" else {}
        self.pool = ref.random_pool(pkv.Pool(nblk, hkv, d, **kw), seed)
        self.bt = ref.tables(rng, self.ctx, nblk, width)
        self.q = torch.randn((self.T, hq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        self.scale = d ** -0.5
        self.sum = pkv.BlockSummary(self.pool)

    def summarize(self, pos=None, cu=None):
        """Bounds of all blocks (one position a block), or of the given positions'."""
        if pos is None:
            pos = np.concatenate([np.arange(0, c, 16) for c in self.ctx]).astype(np.int32)
            cu = np.concatenate([[0], np.cumsum([(c + 15) // 16 for c in self.ctx])]).astype(np.int32)
        pkv.pkv_summarize(self.pool, self.sum, ref.dev(self.bt), ref.dev(cu), ref.dev(pos), ref.dev(self.ctx))
        torch.cuda.synchronize()

    def check_bounds(self):
        K = raw_k(self.pool)
        codes, exps = self.sum.codes.cpu().numpy(), self.sum.exps.cpu().numpy()
        for r, ctx in enumerate(self.ctx):
            for j in range((ctx + 15) // 16):
                b = self.bt[r, j]
                if b < 0 or b >= self.pool.num_blocks:
                    continue
                for g in range(self.hkv):
                    c, e = bounds_of(K[b, g, :min(16, ctx - 16 * j)])
                    assert exps[b, g] == e and np.array_equal(codes[b, g], c), (r, j, g)

    def select(self, k, sinks, recent, **kw):
        return pkv.pkv_select_blocks(self.pool, self.sum, self.q, ref.dev(self.pos), ref.dev(self.bt), ref.dev(self.cu),
                                     k, sinks=sinks, recent=recent, **kw)

    def check_select(self, sel, k, sinks, recent):
        sel = sel.cpu().numpy()
        codes, exps = self.sum.codes.cpu().numpy().astype(np.int64), self.sum.exps.cpu().numpy().astype(np.int64)
        q = self.q.float().double().cpu().numpy()
        for r in range(len(self.ctx)):
            for t in range(self.cu[r], self.cu[r + 1]):
                ids = self.bt[r, :self.pos[t] // 16 + 1]
                valid = (ids >= 0) & (ids < self.pool.num_blocks)
                at = np.where(valid, ids, 0)
                for g in range(self.hkv):
                    s = scores(q[t, g * self.g:(g + 1) * self.g], codes[at, g], exps[at, g])
                    assert np.array_equal(sel[t, g], choose(s, valid, k, sinks, recent)), (r, t, g)

    def attend(self, sel, **kw):
        return pkv.pkv_sparse_attn(self.pool, self.q, ref.dev(self.pos), ref.dev(self.bt), ref.dev(self.cu), sel,
                                   self.scale, **kw)

    def check_attend(self, sel, o, lse):
        torch.cuda.synchronize()
        K, V = ref.pool_values(self.pool, "k"), ref.pool_values(self.pool, "v")
        sel, o, lse = sel.cpu().numpy(), o.float().cpu().numpy(), lse.cpu().numpy()
        q = self.q.float().double().cpu().numpy()
        for r in range(len(self.ctx)):
            for t in range(self.cu[r], self.cu[r + 1]):
                p = int(self.pos[t])
                for g in range(self.hkv):
                    blocks = [b for b in sel[t, g] if 0 <= b <= p // 16 and b < self.bt.shape[1]
                              and 0 <= self.bt[r, b] < self.pool.num_blocks]
                    ids = self.bt[r, blocks]
                    slot = (np.array(blocks, np.int64)[:, None] * 16 + np.arange(16)).reshape(-1)
                    seen = np.repeat((slot <= p)[None], self.g, 0)
                    rows = q[t, g * self.g:(g + 1) * self.g]
                    want, wl, to, tl = ref.softmax_rows(rows, K[ids, g].reshape(-1, self.d), V[ids, g].reshape(-1, self.d),
                                                        seen, self.scale, self.pool.dtype != "bf16")
                    ref.assert_close(o[t, g * self.g:(g + 1) * self.g], want, to, f"O {t} {g}")
                    ref.assert_close(lse[t, g * self.g:(g + 1) * self.g], wl, tl, f"LSE {t} {g}")

    def whole(self, k, sinks, recent):
        self.summarize()
        self.check_bounds()
        sel = self.select(k, sinks, recent)
        torch.cuda.synchronize()
        self.check_select(sel, k, sinks, recent)
        o, lse = self.attend(sel)
        self.check_attend(sel, o, lse)
        assert pkv.pkv_check_device_errors(self.pool) == 0


SMALL = [(1, [0]), (16, [15]), (17, [16]), (40, [0, 20, 39]), (0, []), (500, [499, 100]), (333, list(range(320, 333)))]


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 2, 64), (4, 4, 128), (8, 1, 128), (15, 3, 128), (64, 2, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_small(hq, hkv, d, dtype):
    Case(hq + d, SMALL, hq, hkv, d, dtype).whole(7, 1, 2)


@pytest.mark.parametrize("k,sinks,recent", [(1, 0, 0), (1, 1, 1), (3, 2, 5), (4, 0, 0), (64, 1, 1), (200, 300, 0), (33, 0, 1)])
def test_counts_and_forced_blocks(k, sinks, recent):
    Case(k + sinks, [(1500, [1499]), (70, [69, 5]), (900, [600])], 8, 2, 64).whole(k, sinks, recent)


def test_long_contexts_take_clusters():
    Case(30, [(41000, [40999])], 2, 2, 64).whole(64, 1, 2)
    Case(31, [(20003, [20002, 17])], 8, 1, 128, "fp8_e4m3").whole(128, 0, 1)
    Case(32, [(9000, [8999])], 128, 1, 128).whole(40, 1, 1)


def test_many_tokens():
    rng = np.random.default_rng(33)
    reqs = [(int(c), [int(c) - 1] if c else []) for c in rng.integers(0, 200, 300)]
    Case(33, reqs, 4, 2, 64).whole(5, 1, 1)


def test_scores_that_tie_go_to_the_lower_block():
    c = Case(34, [(1600, [1599])], 4, 1, 64)
    c.pool.k[:] = c.pool.k[:1]                         # every block the same keys
    c.whole(9, 0, 0)
    assert c.select(9, 0, 0)[0, 0].tolist() == list(range(9))
    assert c.select(9, 1, 2)[0, 0].tolist() == list(range(7)) + [98, 99]
    c.pool.k.zero_()
    c.whole(9, 0, 0)
    c.q.zero_()
    c.whole(9, 0, 0)


def test_values_of_every_size():
    """Keys from subnormal to the largest, NaN and infinities; queries with elements that are not finite."""
    c = Case(35, [(640, [639, 320])], 6, 2, 64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    size = torch.exp2(torch.randint(-133, 127, (c.pool.num_blocks, 2, 1, 1), generator=gen, device="cuda").float())
    c.pool.k.copy_((c.pool.k.float() * size).to(torch.bfloat16))
    c.pool.k[3, 0, 2, 5] = float("nan")
    c.pool.k[4, 1, :, 6] = float("nan")
    c.pool.k[5, 0, 1, 7] = float("inf")
    c.pool.k[6, 0, 1, 8] = float("-inf")
    c.pool.k[7] = float("nan")
    c.q[0, 1, 3] = float("inf")
    c.q[0, 4, 9] = float("nan")
    c.q[1] *= 1e-20
    c.summarize()
    c.check_bounds()
    for k in (3, 17):
        c.check_select(c.select(k, 1, 1), k, 1, 1)
    c.q[1] *= 1e-20                                    # below 2^-100: counts as zero
    c.check_select(c.select(9, 0, 1), 9, 0, 1)


def test_bounds_follow_an_append():
    c = Case(36, [(60, list(range(33, 60))), (200, [199]), (16, list(range(16))), (100, [90, 40, 41, 99])], 8, 2, 128)
    c.summarize()
    new_k = torch.randn((c.T, 2, 128), device="cuda").to(torch.bfloat16) * 3
    pkv.pkv_append(c.pool, ref.dev(c.bt), ref.dev(c.cu), ref.dev(c.pos), new_k, new_k)
    c.summarize(c.pos, c.cu)
    c.check_bounds()


def test_the_bound_holds():
    """The score is an upper bound of the group's summed scores of every key, up to the query's own rounding."""
    c = Case(37, [(800, [799])], 8, 2, 128)
    c.summarize()
    K = raw_k(c.pool)
    q = c.q.float().double().cpu().numpy()[0]
    codes, exps = c.sum.codes.cpu().numpy().astype(np.int64), c.sum.exps.cpu().numpy().astype(np.int64)
    for g in range(2):
        qg = q[g * 4:g * 4 + 4]
        f = unit(np.abs(qg).max(), 32767 // 4, -300)
        s = scores(qg, codes[c.bt[0], g], exps[c.bt[0], g]) * 2.0 ** f
        top = (np.rint(qg / 2.0 ** f) * 2.0 ** f).sum(0) @ K[c.bt[0], g].transpose(0, 2, 1)
        assert (top.max(1) <= s * (1 + np.sign(s) * 2.0 ** -23)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_lists_of_the_callers_own(dtype):
    """Any order, padding, blocks behind the token, nothing at all; NaN in what is not seen."""
    c = Case(38, [(300, [299, 130]), (50, [40])], 8, 2, 128, dtype)
    nan = 0x7F if dtype != "bf16" else float("nan")
    for x in (c.pool.k, c.pool.v):
        x[int(c.bt[0, 18]), :, 12:] = nan              # behind the context
        x[int(c.bt[1, 2]), :, 9:] = nan                # behind the token
    sel = np.full((3, 2, 6), -1, np.int32)
    sel[0, 0], sel[0, 1] = [18, 0, -1, 7, -5, 3], [18, 1, 2, 3, 4, 5]
    sel[1, 0] = [18, 17, 9, 8, 2, -1]                  # token at 130: blocks up to 8
    sel[2, 1] = [-1, 2, -1, -1, -1, 0]
    sel = ref.dev(sel)
    o, lse = c.attend(sel)
    c.check_attend(sel, o, lse)
    assert torch.isfinite(o.float()).all() and torch.isinf(lse[1, 4:]).all() and (o[1, 4:] == 0).all()
    assert pkv.pkv_check_device_errors(c.pool) == 0


def test_bad_ids_and_positions_are_flagged_and_skipped():
    c = Case(39, [(300, [299]), (50, [49])], 8, 2, 64)
    c.summarize()
    c.bt[0, 3] = -1
    c.bt[0, 9] = c.pool.num_blocks
    sel = c.select(12, 1, 1)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_BLOCK_ID
    c.check_select(sel, 12, 1, 1)
    assert c.select(19, 1, 1)[0, 0].tolist() == [b for b in range(19) if b not in (3, 9)] + [-1, -1]
    pkv.pkv_check_device_errors(c.pool)
    everything = ref.dev(np.tile(np.arange(19, dtype=np.int32), (2, 2, 1)))
    o, lse = c.attend(everything)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_BLOCK_ID
    c.check_attend(everything, o, lse)
    c.pos[1] = c.bt.shape[1] * 16
    sel = c.select(5, 1, 1)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_POSITION
    assert (sel[1] == -1).all()
    c.summarize(np.array([299, 50], np.int32), np.array([0, 1, 2], np.int32))
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_POSITION


def test_rows_behind_the_last_request_are_left_alone():
    c = Case(40, [(90, [89, 3]), (20, [19])], 8, 2, 64, extra_tokens=6)
    c.summarize()
    sel = torch.full((c.T, 2, 4), 55, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(c.q, 7.0), torch.full((c.T, 8), 3.0, device="cuda")
    c.select(4, 1, 1, out=sel)
    c.attend(sel, out=out, lse=lse)
    c.check_select(sel, 4, 1, 1)
    c.check_attend(sel, out, lse)
    assert (sel[3:] == 55).all() and (out[3:] == 7.0).all() and (lse[3:] == 3.0).all()


def test_captured_step_follows_positions_and_tables():
    c = Case(41, [(700, [699]), (400, [399]), (160, [159])], 16, 2, 128)
    c.summarize()
    bt, cu, pos, ctx = (ref.dev(x) for x in (c.bt, c.cu, c.pos, c.ctx))
    sel = torch.zeros((3, 2, 8), dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(c.q), torch.zeros((3, 16), device="cuda")

    def step():
        pkv.pkv_summarize(c.pool, c.sum, bt, cu, pos, ctx)
        pkv.pkv_select_blocks(c.pool, c.sum, c.q, pos, bt, cu, 8, sinks=1, recent=2, out=sel)
        pkv.pkv_sparse_attn(c.pool, c.q, pos, bt, cu, sel, c.scale, out=out, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        c.pos = np.array([600 - 37 * k, 399 - k, 16 + k], np.int32)
        pos.copy_(ref.dev(c.pos))
        c.q.copy_(torch.randn(c.q.shape, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        c.check_select(sel, 8, 1, 2)
        c.check_attend(sel, out, lse)


def test_all_blocks_selected_equals_the_causal_attention():
    """A selection that covers the context attends as pkv_paged_attn does: twice the bound, once for each."""
    c = Case(42, [(333, [332]), (64, [63])], 8, 2, 128)
    c.summarize()
    sel = c.select(21, 1, 1)
    o, lse = c.attend(sel)
    c.check_attend(sel, o, lse)
    meta = pkv.HostMeta(c.cu, c.ctx, c.pos)
    po, pl = pkv.pkv_paged_attn(c.pool, c.q, ref.dev(c.pos), ref.dev(c.bt), ref.dev(c.ctx), ref.dev(c.cu), meta, c.scale)
    torch.cuda.synchronize()
    c.check_attend(sel, po, pl)


def test_refusals():
    c = Case(44, [(100, [99])], 8, 2, 64)
    pos, bt, cu = ref.dev(c.pos), ref.dev(c.bt), ref.dev(c.cu)
    sel = c.select(4, 1, 1)
    with pytest.raises(ValueError):
        c.select(0, 1, 1)
    for sinks, recent in ((-1, 0), (0, -1)):
        with pytest.raises(pkv.PkvError) as e:
            c.select(4, sinks, recent)
        assert e.value.code == pkv.PKV_EINVAL
    p, lib = c.q.data_ptr(), pkv.load_library()
    for k in (0, -1, (1 << 27) + 1):
        assert lib.pkv_select_blocks(c.pool.handle, p, 8, p, p, 7, p, 1, 1, p, p, k, 1, 1, p, p, 1 << 30, None) == pkv.PKV_EINVAL
        assert lib.pkv_sparse_attn(c.pool.handle, p, 8, p, p, 7, p, 1, 1, p, k, 0.1, p, None, p, 1 << 30, None) == pkv.PKV_EINVAL
    c.scale = 0.0
    with pytest.raises(pkv.PkvError, match="scale"):
        c.attend(sel)
    c.scale = 0.1
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError, match="workspace"):
        c.attend(sel, workspace=small)
    with pytest.raises(ValueError):
        pkv.BlockSummary(c.pool, codes=c.sum.codes)
    with pytest.raises(ValueError):
        pkv.BlockSummary(c.pool, c.sum.codes[:, :1].contiguous(), c.sum.exps)
    with pytest.raises(TypeError):
        pkv.BlockSummary(c.pool, c.sum.codes.float(), c.sum.exps)
    for kw in (dict(q_positions=ref.dev(np.zeros(2, np.int32))), dict(block_tables=torch.cat([bt, bt])),
               dict(selected=sel[:, :1].contiguous())):
        args = dict(q_positions=pos, block_tables=bt, cu_q_lens=cu, selected=sel)
        args.update(kw)
        with pytest.raises(ValueError):
            pkv.pkv_sparse_attn(c.pool, c.q, scale=0.1, **args)


def test_no_tokens_is_nothing_to_do():
    c = Case(45, [(100, [99])], 8, 2, 64)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_summarize(c.pool, c.sum, e.view(0, 3), zero, e, e)
    sel = pkv.pkv_select_blocks(c.pool, c.sum, c.q[:0], e, e.view(0, 3), zero, 5)
    o, lse = pkv.pkv_sparse_attn(c.pool, c.q[:0], e, e.view(0, 3), zero, sel, 0.1)
    assert sel.shape == (0, 2, 5) and o.shape == (0, 8, 64) and lse.shape == (0, 8)
    assert pkv.pkv_check_device_errors(c.pool) == 0


def test_tokens_in_parts():
    """More tokens than the workspace holds the scores of at a time."""
    c = Case(46, [(300, list(range(100, 300)))], 2, 2, 64, width=100_000)     # 80 tokens a part
    c.bt[:, 19:] = -1
    c.whole(6, 1, 1)


def test_heads_that_fill_no_octet():
    for hkv in (3, 5, 7, 9, 12, 20):
        Case(hkv, [(700, [699]), (90, [89, 5])], hkv * 2, hkv, 64 if hkv % 2 else 128).whole(9, 1, 1)


def test_many_groups_and_long_lists():
    rng = np.random.default_rng(47)
    reqs = [(int(n), [int(n) - 1]) for n in rng.integers(600, 2500, 70)]
    Case(47, reqs, 16, 8, 64, "fp8_e4m3").whole(40, 1, 1)        # a share a warp
    for dtype, d in (("bf16", 64), ("bf16", 128), ("fp8_e4m3", 64), ("fp8_e4m3", 128)):
        Case(48, reqs[:25], 16, 8, d, dtype).whole(40, 1, 1)     # a CTA of six warps a group
        Case(48, reqs[:9], 16, 8, d, dtype).whole(40, 1, 1)      # of twelve
    Case(48, reqs[:25], 16, 8, 64).whole(70, 1, 1)               # of four
    Case(49, reqs[:3], 16, 8, 128).whole(90, 1, 1)               # shares of CTAs


def test_blocks_beyond_4_gb():
    c = Case(50, [(700, [699]), (40, [20])], 8, 2, 128)
    nb, small = 600_000, c.pool
    pool = pkv.Pool(nb, 2, 128)
    pool.k[nb - small.num_blocks:] = small.k
    pool.v[nb - small.num_blocks:] = small.v
    low, low_bt = c.sum, c.bt
    c.pool, c.sum = pool, pkv.BlockSummary(pool)
    c.bt = np.where(c.bt >= 0, c.bt + nb - small.num_blocks, -1).astype(np.int32)
    c.summarize()
    sel = c.select(11, 1, 1)
    o, lse = c.attend(sel)
    torch.cuda.synchronize()
    assert pkv.pkv_check_device_errors(pool) == 0
    tail = pkv.BlockSummary(small, c.sum.codes[nb - small.num_blocks:].contiguous(), c.sum.exps[nb - small.num_blocks:].contiguous())
    c.pool, c.sum, c.bt = small, tail, low_bt
    c.check_bounds()
    c.check_select(sel, 11, 1, 1)
    c.check_attend(sel, o, lse)
    pool.close()


@pytest.mark.parametrize("hq,hkv,d,dtype", [(2, 2, 64, "bf16"), (8, 2, 128, "bf16"), (24, 3, 64, "bf16"), (5, 5, 128, "fp8_e4m3"),
                                            (16, 8, 128, "bf16"), (12, 12, 64, "fp8_e4m3"), (128, 1, 128, "bf16"),
                                            (80, 20, 128, "fp8_e4m3")])
def test_small_batches_in_wide_tables(hq, hkv, d, dtype):
    """The kernels of large batches on the sizes of small ones: as pairs of tokens, and one by one."""
    Case(51, SMALL, hq, hkv, d, dtype, width=600).whole(7, 1, 1)
    Case(52, [(40, [39]), (700, [699]), (17, [16]), (300, [299, 298, 297])], hq, hkv, d, dtype, width=600).whole(7, 1, 1)


def test_many_heads():
    Case(53, [(300, list(range(290, 300))), (40, [39, 38])], 130, 65, 64, width=600).whole(6, 1, 1)
    Case(56, [(100, [99])], 301, 301, 64, width=600).whole(3, 1, 1)
    Case(57, [(100, [99, 98])], 600, 300, 64).whole(3, 1, 1)


def test_query_heads_beyond_the_staging_rows():
    Case(54, [(300, [299, 298]), (40, [39, 38])], 200, 40, 64, width=600).whole(6, 1, 1)      # 13 of 40 heads staged
    Case(55, [(300, [299]), (40, [39])], 200, 2, 64, width=600).whole(6, 1, 1)                # none
