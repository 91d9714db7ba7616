"""Attention with modified scores and masks, through the C ABI, against its formulas in 64 bits (score_ref)."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import score_ref
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "fp8_e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def make_pool(nb, hkv, d, dtype, seed):
    if dtype != "int8":
        scales = dict(k_scale=0.03, v_scale=0.5) if dtype == "fp8_e4m3" else {}
        return ref.random_pool(pkv.Pool(nb, hkv, d, dtype=dtype, **scales), seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool = pkv.Pool(nb, hkv, d, dtype="int8")
    for x, e in ((pool.k, pool.k_exps), (pool.v, pool.v_exps)):
        x.copy_((torch.randn(x.shape, generator=gen, device="cuda") * 36).round().clamp(-127, 127))
        e.copy_(torch.randint(-7, -3, e.shape, generator=gen, device="cuda"))
    return pool


def values(pool, which):
    if pool.dtype != "int8":
        return ref.pool_values(pool, which)
    e = getattr(pool, which + "_exps").cpu().numpy().astype(np.int64)
    return np.ldexp(getattr(pool, which).cpu().numpy().astype(np.float64), np.clip(e, -126, 121)[:, :, None, None])


class Case:
    """reqs: (context, query positions)."""

    def __init__(self, seed, reqs, hq, hkv, d, dtype="bf16", extra=0, width=None, **opts):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.g, self.extra = hq, hkv, d, hq // hkv, extra
        self.ctx = np.array([r[0] for r in reqs], np.int32)
        self.cu = np.cumsum([0] + [len(r[1]) for r in reqs]).astype(np.int32)
        self.pos = np.concatenate([np.asarray(r[1], np.int32) for r in reqs] + [np.full(extra, 3, np.int32)]).astype(np.int32)
        nb = int(sum((c + 15) // 16 for c in self.ctx)) + 4
        self.pool = make_pool(nb, hkv, d, dtype, seed)
        self.bt = ref.tables(rng, self.ctx, nb, width)
        self.q = torch.tensor(rng.standard_normal((len(self.pos), hq, d)), dtype=torch.float32).to(torch.bfloat16)
        self.scale = float(np.float32(opts.get("scale", d ** -0.5)))
        self.cap, self.window = opts.get("softcap", 0.0), opts.get("window", 0)
        self.slopes = np.float32(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)) if opts.get("slopes") else None
        self.prefix = np.asarray(opts["prefix"], np.int32) if "prefix" in opts else None
        self.first = None
        if opts.get("docs"):
            self.first = np.maximum(self.pos - rng.integers(0, opts["docs"], len(self.pos)), -1).astype(np.int32)
            self.first[::7] = self.pos[::7] + 1          # some tokens see nothing but the prefix
        self.seen_empty = False

    def call(self, **kw):
        opt = lambda x: None if x is None else ref.dev(x)
        return pkv.pkv_score_attn(self.pool, self.q.cuda(), ref.dev(self.pos), ref.dev(self.bt), ref.dev(self.ctx),
                                  ref.dev(self.cu), self.scale, softcap=self.cap, window=self.window,
                                  slopes=opt(self.slopes), first_keys=opt(self.first), prefix_lens=opt(self.prefix), **kw)

    def check(self, o, lse, tokens=None):
        o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
        k, v = values(self.pool, "k"), values(self.pool, "v")
        q = self.q.double().numpy()
        for r in range(len(self.ctx)):
            ctx = int(self.ctx[r])
            pre = 0 if self.prefix is None else int(self.prefix[r])
            for g in range(self.hkv):
                kk, there = ref.gather(k, self.bt[r], ctx, g)
                vv, _ = ref.gather(v, self.bt[r], ctx, g)
                hs = slice(g * self.g, (g + 1) * self.g)
                for t in range(self.cu[r], self.cu[r + 1]):
                    if tokens is not None and t not in tokens:
                        continue
                    seen = score_ref.sees(int(self.pos[t]), ctx, pre, 0 if self.first is None else int(self.first[t]),
                                          self.window) & there
                    want, wl, tol, tl = score_ref.rows(q[t, hs], kk, vv, int(self.pos[t]), seen, self.scale, self.cap,
                                                       None if self.slopes is None else self.slopes[hs].astype(np.float64),
                                                       self.pool.dtype == "fp8_e4m3")
                    self.seen_empty |= not seen.any()
                    ref.assert_close(o[t, hs], want, tol, f"O of token {t}, KV head {g}")
                    ref.assert_close(lse[t, hs], wl, tl, f"LSE of token {t}, KV head {g}")

    def run(self, **kw):
        out = torch.full(self.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 5.0, device="cuda")
        o, l = self.call(out=out, lse=lse, **kw)
        assert o is out and l is lse
        self.check(o, l)
        last = self.cu[-1]
        assert (o[last:] == 5.0).all() and (l[last:] == 5.0).all()
        assert pkv.pkv_check_device_errors(self.pool) == 0
        return self


def tail(ctx, n):
    return ctx, list(range(ctx - n, ctx))


BATCHES = {
    "one": [tail(1, 1)],
    "decode": [tail(c, 1) for c in (1, 15, 16, 17, 33, 130, 700, 1025)],
    "steps": [tail(40, 3), tail(300, 7), tail(16, 2), (0, []), tail(129, 5), tail(2, 2)],
    "prompts": [tail(300, 300), tail(17, 17), tail(1, 1), tail(260, 131)],
    "recompute": [(200, list(range(0, 33)) + list(range(190, 200))), (90, [89, 3, 40, 40])],
}
OPTIONS = {
    "causal": {},
    "cap": dict(softcap=2.0),
    "slopes": dict(slopes=True),
    "window": dict(window=37),
    "window1": dict(window=1, softcap=30.0),
    "docs": dict(docs=60),
    "prefix": dict(prefix="third"),
    "all": dict(softcap=5.0, slopes=True, window=50, docs=200, prefix="few"),
}


def options(name, batch):
    o = dict(OPTIONS[name])
    if "prefix" in o:
        o["prefix"] = [c // 3 if o["prefix"] == "third" else min(c, 4) for c, _ in batch]
    return o


@pytest.fixture(params=[1, 2], ids=["rows", "tiles"])
def form(request, monkeypatch):
    """Which kernel takes the batch."""
    make = make_pool

    def forced(*args):
        pool = make(*args)
        pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, request.param)
        return pool

    monkeypatch.setitem(globals(), "make_pool", forced)
    return request.param


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("opt", list(OPTIONS))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_against_the_formulas(batch, opt, dtype, form):
    reqs = BATCHES[batch]
    Case(len(reqs) + 11, reqs, 8, 2, 64, dtype, extra=2, **options(opt, reqs)).run()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (64, 8, 128), (24, 1, 64), (15, 3, 128), (128, 1, 64), (2, 2, 64), (5, 5, 128)])
@pytest.mark.parametrize("opt", ["causal", "all"])
def test_heads(hq, hkv, d, dtype, opt, form):
    reqs = [tail(150, 2), tail(31, 31), tail(500, 1), tail(64, 40)]
    Case(5, reqs, hq, hkv, d, dtype, extra=1, **options(opt, reqs)).run()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_contexts_cut_into_shares(dtype, form):
    reqs = [tail(30000, 1), tail(17, 1), tail(9001, 2)]
    Case(6, reqs, 8, 2, 128, dtype).run()
    c = Case(7, reqs, 8, 2, 128, dtype, softcap=4.0, slopes=True, window=9000, prefix=[100, 17, 0]).run()
    c.window = 130
    c.run()


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_requests(dtype, form):
    rng = np.random.default_rng(4)
    reqs = [tail(int(c), 1) for c in rng.integers(1, 90, 700)]
    Case(8, reqs, 4, 2, 64, dtype, window=20).run()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("opt", ["causal", "cap", "slopes", "all"])
def test_prompts_of_several_tiles(dtype, opt):
    """The chosen form (tiles): pairs and single tiles over many key tiles, groups cut into shares."""
    reqs = [tail(1500, 700), tail(900, 900), tail(40, 1)]
    Case(19, reqs, 8, 2, 128, dtype, extra=3, **options(opt, reqs)).run()


def test_empty_rows_are_zero(form):
    c = Case(9, BATCHES["steps"], 4, 2, 64, docs=5)
    c.run()
    assert c.seen_empty


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_values_that_are_not_finite(dtype, form):
    """Infinite and NaN keys and values reach the rows that see them, and no others."""
    reqs = [tail(70, 40), tail(300, 3)]
    c = Case(10, reqs, 8, 2, 64, dtype, window=30, prefix=[5, 0])
    bad = [float("inf"), float("-inf"), float("nan")] if dtype == "bf16" else [float("nan")] * 3
    for i, x in enumerate(bad):
        for which, pos in (("k", 20 + i), ("v", 44 + 2 * i), ("v", 3)):
            p = getattr(c.pool, which)
            at = (c.bt[0][pos // 16], i % 2, pos % 16, 7 * i + 1)
            if dtype == "bf16":
                p[at] = x
            else:
                p[at] = 0x7f
    # stale values behind the contexts, and in a block of nobody
    for p in (c.pool.k, c.pool.v):
        stale = float("nan") if dtype == "bf16" else 0x7f
        p[c.bt[0][4], :, 70 - 64:] = stale
        p[c.bt[1][18], :, 300 - 288:] = stale
    o, lse = c.call()
    # a row that sees a key that is not finite: by its formula where that has a value, else merely not finite
    k, v = values(c.pool, "k"), values(c.pool, "v")
    clean = []
    for r in range(2):
        for t in range(c.cu[r], c.cu[r + 1]):
            seen = score_ref.sees(int(c.pos[t]), int(c.ctx[r]), int(c.prefix[r]), 0, 30)
            hit = False
            for g in range(2):
                kk, _ = ref.gather(k, c.bt[r], int(c.ctx[r]), g)
                vv, _ = ref.gather(v, c.bt[r], int(c.ctx[r]), g)
                for h in range(g * 4, g * 4 + 4):
                    dims = ~np.isfinite(vv[seen]).all(0)
                    got = o[t, h].float().cpu().numpy()
                    if not np.isfinite(kk[seen]).all():
                        hit = True
                        assert not np.isfinite(got).all() or not np.isfinite(lse[t, h].item())
                    elif dims.any():
                        hit = True
                        assert (~np.isfinite(got) == dims).all()
                    else:
                        assert np.isfinite(got).all()
            if not hit:
                clean.append(t)
    assert clean and len(clean) < c.cu[-1]
    c.check(o, lse, set(clean))


def test_exponents_of_int8_pages(form):
    """The largest and smallest exponents, and pages whose exponents were never written."""
    reqs = [tail(64, 3), tail(40, 1)]
    c = Case(11, reqs, 4, 2, 64, "int8")
    c.pool.v_exps[c.bt[0][0]] = 40
    c.pool.v_exps[c.bt[0][1]] = -126
    c.pool.k_exps[c.bt[0][2]] = -126
    c.pool.k_exps[c.bt[1][0]] = -40
    c.run()
    out = c.call()
    other = [i for i in range(c.pool.num_blocks) if i not in c.bt]
    c.pool.v_exps[other] = 127
    c.pool.k_exps[other] = -128
    again = c.call()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


def test_extreme_scores(form):
    """Scores far beyond the cap, a large scale, distances past 2^24 steps of a float."""
    reqs = [tail(50, 50)]
    Case(12, reqs, 4, 2, 64, softcap=30.0, scale=50.0).run()
    Case(13, reqs, 4, 2, 64, scale=3.0).run()
    c = Case(14, reqs, 4, 2, 64, slopes=True)
    c.slopes = np.array([100.0, -0.25, 0.0, 1e-3], np.float32)
    c.run()


def test_bad_blocks_lengths_and_positions(form):
    reqs = [tail(100, 3), tail(40, 2), tail(33, 1)]
    c = Case(15, reqs, 8, 2, 64, prefix=[20, 0, 0], window=30)
    c.bt[0, 5], c.bt[1, 1] = -1, c.pool.num_blocks
    o, lse = c.call()
    c.check(o, lse)
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_BLOCK_ID
    c = Case(15, reqs, 8, 2, 64, prefix=[20, 0, 0])
    c.bt[0, 3] = -7
    c.pos[0], c.pos[3], c.pos[5] = -5, 2 ** 31 - 1, -2 ** 31
    o, lse = c.call()
    c.check(o, lse)
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_BLOCK_ID | pkv.PKV_DEVERR_POSITION
    c = Case(15, reqs, 8, 2, 64, prefix=[20, 0, 0])
    c.ctx[1], c.prefix[2] = 5000, 34
    c.call()
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_POSITION
    c = Case(15, reqs, 8, 2, 64)
    c.cu[:] = [-3, 2, 4, 999]
    c.call()
    assert pkv.pkv_check_device_errors(c.pool) & pkv.PKV_DEVERR_POSITION


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_step_of_an_8_bit_cache(dtype):
    """The new rows are appended, attended to and read back: the run of calls of a decoding step."""
    rng = np.random.default_rng(16)
    reqs = [tail(100, 2), tail(17, 1), tail(48, 16)]
    c = Case(16, reqs, 8, 2, 64, dtype, softcap=20.0)
    k, v = (torch.tensor(rng.standard_normal((19, 2, 64)), dtype=torch.float32).to(torch.bfloat16).cuda() for _ in range(2))
    d = ref.dev
    if dtype == "int8":
        pkv.pkv_append_int8(c.pool, d(c.bt), d(c.cu), d(c.pos), d(np.array([98, 16, 32], np.int32)), k, v)
    else:
        pkv.pkv_append(c.pool, d(c.bt), d(c.cu), d(c.pos), k, v)
    o, lse = c.call()
    kr, _ = pkv.pkv_read_rows(c.pool, d(c.bt), d(c.cu), d(c.pos))
    c.check(o, lse)
    if dtype == "bf16":
        assert torch.equal(kr, k)
    elif dtype == "int8":
        # Half a step of 2^e, ties included (x = -33.5 * 2^-4 is off by exactly that much): 2^e by ldexp, which is exact, not
        # by pow, which on the device is not.
        e = c.pool.k_exps[torch.as_tensor(np.repeat([c.bt[0][6], c.bt[1][1], c.bt[2][2]], [2, 1, 16])).long()].cpu().numpy()
        step = torch.as_tensor(np.ldexp(1.0, e.astype(np.int64))).cuda()
        assert ((kr.double() - k.double()).abs() <= 0.5 * step[:, :, None]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_graph_streams_and_devices(dtype, form):
    """Captured once, replayed with other lengths, tables, positions and masks; on another stream; bits do not change."""
    reqs = [tail(200, 3), tail(77, 2)]
    a, b = (Case(17 + i, rq, 8, 2, 64, dtype, extra=1, window=40, softcap=8.0, prefix=pre, docs=90)
            for i, (rq, pre) in enumerate([(reqs, [3, 0]), ([tail(31, 1), tail(260, 4)], [0, 20])]))
    assert a.pool.num_blocks >= 4
    width = max(a.bt.shape[1], b.bt.shape[1])
    wide = lambda x: np.pad(x, ((0, 0), (0, width - x.shape[1])), constant_values=-1)
    nb = max(a.pool.num_blocks, b.pool.num_blocks)
    pool = make_pool(nb, 2, 64, dtype, 3)
    for c in (a, b):
        c.pool, c.bt = pool, wide(c.bt)
    st = {n: ref.dev(getattr(a, n)) for n in ("pos", "bt", "ctx", "cu", "first", "prefix")}
    q = a.q.cuda()
    go = lambda **kw: pkv.pkv_score_attn(pool, q, st["pos"], st["bt"], st["ctx"], st["cu"], a.scale, softcap=8.0, window=40,
                                         first_keys=st["first"], prefix_lens=st["prefix"], **kw)
    want = go()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o, lse = go()
    for c in (a, b, a):
        for n, x in st.items():
            x.copy_(ref.dev(getattr(c, n)))
        q.copy_(c.q)
        g.replay()
        torch.cuda.synchronize()
        c.check(o[:5], lse[:5])
    assert torch.equal(o[:5], want[0][:5]) and torch.equal(lse[:5], want[1][:5])
    s.wait_stream(torch.cuda.current_stream())
    x, y = go(stream=s)
    with torch.cuda.stream(s):
        z, w = go()
    s.synchronize()
    for i, j in ((x, y), (z, w)):
        assert torch.equal(i[:5], want[0][:5]) and torch.equal(j[:5], want[1][:5])
    assert go(want_lse=False)[1] is None
    assert pkv.pkv_check_device_errors(pool) == 0


def test_refusals():
    c = Case(18, [tail(20, 2)], 4, 2, 64)
    assert c.call()[0].shape == (2, 4, 64)
    for kw in (dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-30), dict(window=-1),
               dict(scale=0.0), dict(scale=float("inf"))):
        d = Case(18, [tail(20, 2)], 4, 2, 64)
        for n, x in kw.items():
            setattr(d, n, x)
        with pytest.raises(pkv.PkvError) as e:
            d.call()
        assert e.value.code == pkv.PKV_EINVAL
    need = pkv.pkv_score_attn_workspace_size(c.pool, 4, 2, 1, 2)
    for ws in (torch.empty(need - 256, dtype=torch.uint8, device="cuda"), torch.empty(need + 256, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(pkv.PkvError) as e:
            c.call(workspace=ws)
        assert e.value.code == pkv.PKV_EINVAL
    c.slopes = np.zeros(3, np.float32)
    with pytest.raises(ValueError):
        c.call()
    c.slopes = np.zeros(4, np.float64)
    with pytest.raises(TypeError):
        c.call()
    c.slopes, c.first = None, np.zeros(3, np.int32)
    with pytest.raises(ValueError):
        c.call()
    c.first, c.prefix = None, np.zeros(2, np.int32)
    with pytest.raises(ValueError):
        c.call()
    big = pkv.Pool(4, 1, 64)
    q = torch.zeros((1, 129, 64), dtype=torch.bfloat16, device="cuda")
    i = lambda *x: ref.dev(np.array(x, np.int32))
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_score_attn(big, q, i(0), i(0).view(1, 1), i(1), i(0, 1), 1.0)
    assert e.value.code == pkv.PKV_EUNSUPPORTED
    z = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = pkv.pkv_score_attn(big, z, i(), i(0).view(1, 1), i(0), i(0, 0), 1.0)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
