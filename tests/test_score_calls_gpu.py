"""Attention with modified scores, and reading rows back, in the calls that their documentation allows: waits that run out,
streams and threads side by side, graphs that share a workspace, values that are not finite, outputs of any alignment."""
import threading

import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv
from test_score_gpu import DTYPES, Case, built, make_pool, tail, values  # noqa: F401

pytestmark = pytest.mark.gpu


def forced(case, form):
    pkv.pkv_debug_set(case.pool, pkv.PKV_DEBUG_TREE_FORM, form)
    return case


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_wait_that_runs_out_is_reported_and_the_pool_recovers(d, dtype):
    """(The rows form waits on no barrier.)"""
    c = forced(Case(40, [tail(1500, 70), tail(300, 33), tail(40, 3)], 8, 2, d, dtype), 2)
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WAIT_LIMIT_NS, 2_000_000)
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WITHHOLD_COPY, 2)
    c.call()
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_TIMEOUT
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WITHHOLD_COPY, 0)
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_WAIT_LIMIT_NS, 1_000_000_000)
    c.run()


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_calls_side_by_side(dtype, form):
    """Two streams, and two threads, each with batches of its own over pools of its own; then one pool from two streams."""
    cases = [forced(Case(50 + i, [tail(900 + 200 * i, 5 + i), tail(64, 1)], 8, 2, 64, dtype, softcap=3.0), form) for i in range(2)]
    want = [c.call() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(10):
                    got[i].append(cases[i].call())
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 10
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    outs = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(cases[0].call())
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    assert all(pkv.pkv_check_device_errors(c.pool) == 0 for c in cases)


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
def test_graphs_that_share_a_workspace(form):
    """Replayed one after the other in any order: nothing of one call is left for the next."""
    pool = make_pool(140, 2, 64, "int8", 60)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, form)
    cases = [Case(61 + i, r, 8, 2, 64, "int8", **o) for i, (r, o) in enumerate([
        ([tail(1900, 9)], dict(slopes=True)), ([tail(700, 130), tail(33, 2), tail(500, 1)], dict(softcap=4.0, window=100))])]
    for c in cases:
        c.pool = pool
        c.bt %= 140
    need = max(pkv.pkv_score_attn_workspace_size(pool, 8, c.bt.shape[1], len(c.ctx), len(c.pos)) for c in cases)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    graphs, outs, keep = [], [], []
    for c in cases:
        args = [c.q.cuda()] + [ref.dev(x) for x in (c.pos, c.bt, c.ctx, c.cu)]
        slopes = None if c.slopes is None else ref.dev(c.slopes)
        keep.append((args, slopes))
        go = lambda: pkv.pkv_score_attn(pool, *args, c.scale, softcap=c.cap, window=c.window, slopes=slopes, workspace=ws)
        go()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(go())
        graphs.append(g)
    for order in ([0, 1], [1, 0, 0, 1]):
        for o, lse in outs:
            o.fill_(7.0)
            lse.fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for c, (o, lse) in zip(cases, outs):
            c.check(o, lse)


@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_many_values_that_are_not_finite_in_blocks_that_few_rows_see(dtype, form):
    """More than any list of them, several of a dim, of both signs: a row's dim is infinite where all it sees there is of
    one sign, NaN otherwise, finite where it sees none."""
    c = forced(Case(70, [tail(700, 4)], 8, 2, 64, dtype, window=600, prefix=[3]), form)
    rng = np.random.default_rng(71)
    inf, nan = float("inf"), float("nan")
    for pos in (0, 2, 97, 98, 99, 100, 696, 697, 698, 699):      # the prefix, the window's edge, the new tokens
        blk, slot = int(c.bt[0][pos // 16]), pos % 16
        for dim in rng.choice(64, 24, replace=False):
            c.pool.v[blk, :, slot, int(dim)] = 0x7f if dtype != "bf16" else (inf, inf, -inf, nan)[rng.integers(4)]
    o, lse = c.call()
    o = o.float().cpu().numpy()
    v = values(c.pool, "v")
    kinds = set()
    for t in range(4):
        pos = int(c.pos[t])
        seen = [j for j in range(pos + 1) if j < 3 or j > pos - 600]
        for g in range(2):
            vv = np.stack([v[c.bt[0][j // 16], g, j % 16] for j in seen])
            with np.errstate(invalid="ignore"):
                odd = np.where(np.isfinite(vv), 0.0, vv).sum(0)
            for h in range(4 * g, 4 * g + 4):
                for dim in range(64):
                    got = o[t, h, dim]
                    kinds.add(str(odd[dim]))
                    if np.isnan(odd[dim]):
                        assert np.isnan(got)
                    elif np.isinf(odd[dim]):
                        assert got == odd[dim]
                    else:
                        assert np.isfinite(got)
    assert kinds == ({"inf", "-inf", "nan", "0.0"} if dtype == "bf16" else {"nan", "0.0"})
    assert torch.isfinite(lse).all()
    assert pkv.pkv_check_device_errors(c.pool) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_read_back_to_any_16_byte_boundary(dtype):
    pool = make_pool(9, 3, 64, dtype, 80)
    bt = ref.dev(np.array([[4, 1, 7], [2, 8, -1]], np.int32))
    pos = ref.dev(np.array([0, 15, 16, 47, 31, 3], np.int32))
    cu = ref.dev(np.array([0, 4, 6], np.int32))
    want = pkv.pkv_read_rows(pool, bt, cu, pos)
    n = 6 * 3 * 64
    for ka, va in ((0, 8), (8, 0), (8, 8), (16, 16)):            # in values of two bytes
        big = torch.full((2, n + 16 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
        k, v = big[0, ka:ka + n].view(6, 3, 64), big[1, va:va + n].view(6, 3, 64)
        pkv.pkv_read_rows(pool, bt, cu, pos, k_out=k, v_out=v)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        assert (big[0, :ka] == 9).all() and (big[0, ka + n:] == 9).all()
        assert (big[1, :va] == 9).all() and (big[1, va + n:] == 9).all()
    blk = bt.cpu().numpy()
    exact = values(pool, "k")
    for t, p in enumerate([0, 15, 16, 47, 31, 3]):
        row = exact[blk[0 if t < 4 else 1][p // 16], :, p % 16]
        if dtype != "fp8_e4m3":                                   # (codes times a scale are rounded)
            assert np.array_equal(want[0][t].double().cpu().numpy(), row)


def test_more_items_than_are_counted_are_refused():
    pool = pkv.Pool(4, 2, 64)
    for reqs, tokens in ((2 ** 31 - 1, 1), (2 ** 30, 2 ** 30)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_score_attn_workspace_size(pool, 8, 4, reqs, tokens)
        assert e.value.code == pkv.PKV_EUNSUPPORTED
    assert pkv.pkv_score_attn_workspace_size(pool, 8, 4, 1000, 1000) > 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_pools_whose_offsets_pass_32_bits(dtype):
    """Blocks at both ends of a pool whose K and V take more than 2^32 bytes each."""
    hkv, d = 2, 64
    nb = (2 ** 32 + 2 ** 28) // (hkv * 16 * d) // (2 if dtype == "bf16" else 1)
    pool = pkv.Pool(nb, hkv, d, dtype=dtype, **(dict(k_scale=0.03, v_scale=0.5) if dtype == "fp8_e4m3" else {}))
    ends = [nb - 1, 0, nb - 2, 1, nb - 3]
    ctx = 16 * len(ends) - 5
    rng = np.random.default_rng(90)
    bt = np.array([ends], np.int32)
    pos = np.arange(ctx, dtype=np.int32)
    rows = [torch.tensor(rng.standard_normal((ctx, hkv, d)), dtype=torch.float32).to(torch.bfloat16).cuda() for _ in range(2)]
    i = lambda x: ref.dev(np.asarray(x, np.int32))
    if dtype == "int8":
        pkv.pkv_append_int8(pool, i(bt), i([0, ctx]), i(pos), i([0]), *rows)
    else:
        pkv.pkv_append(pool, i(bt), i([0, ctx]), i(pos), *rows)
    small = pkv.Pool(len(ends), hkv, d, dtype=dtype, **(dict(k_scale=0.03, v_scale=0.5) if dtype == "fp8_e4m3" else {}))
    near = np.arange(len(ends), dtype=np.int32)[None]
    if dtype == "int8":
        pkv.pkv_append_int8(small, i(near), i([0, ctx]), i(pos), i([0]), *rows)
    else:
        pkv.pkv_append(small, i(near), i([0, ctx]), i(pos), *rows)
    q = torch.randn((ctx, 4, d), generator=torch.Generator().manual_seed(91)).to(torch.bfloat16).cuda()
    for form in (1, 2):
        got = []
        for p, table in ((pool, bt), (small, near)):
            pkv.pkv_debug_set(p, pkv.PKV_DEBUG_TREE_FORM, form)
            got.append((pkv.pkv_read_rows(p, i(table), i([0, ctx]), i(pos)),
                        pkv.pkv_score_attn(p, q, i(pos), i(table), i([ctx]), i([0, ctx]), 0.125, softcap=3.0, window=50)))
            assert pkv.pkv_check_device_errors(p) == 0
        for a, b in zip(got[0][0] + got[0][1], got[1][0] + got[1][1]):
            assert torch.equal(a, b)
    if dtype == "bf16":
        assert torch.equal(got[0][0][0], rows[0]) and torch.equal(got[0][0][1], rows[1])
