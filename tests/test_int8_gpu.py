"""The 8-bit cache with an exponent for each block: quantising write, reading back, page operations.

Codes, exponents and int8 values read back are whole numbers or exact: equal, not close.
"""
import numpy as np
import pytest
import torch

import attn_ref as ref
from int8_ref import Cache
from paged_kv_attention_25_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def filled(nb, hkv, d, seed):
    """A pool of random codes and moderate exponents."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool = pkv.Pool(nb, hkv, d, dtype="int8")
    for x in (pool.k, pool.v):
        x.copy_(torch.randint(-127, 128, x.shape, generator=gen, device="cuda"))
    for x in (pool.k_exps, pool.v_exps):
        x.copy_(torch.randint(-9, -3, x.shape, generator=gen, device="cuda"))
    return pool


def rows(rng, shape, spread=0.8):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)) * spread)
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def run(pool, bt, cu, pos, held, k, v, stream=None):
    d = ref.dev
    pkv.pkv_append_int8(pool, d(bt), d(np.asarray(cu, np.int32)), d(np.asarray(pos, np.int32)),
                        d(np.asarray(held, np.int32)), k.cuda(), v.cuda(), stream=stream)


def caches(pool):
    return [Cache(c.cpu().numpy(), e.cpu().numpy()) for c, e in ((pool.k, pool.k_exps), (pool.v, pool.v_exps))]


def check(pool, want, kept, untouched):
    torch.cuda.synchronize()
    for c, (codes, exps) in zip(want, ((pool.k, pool.k_exps), (pool.v, pool.v_exps))):
        assert np.array_equal(exps.cpu().numpy(), c.exps)
        got = codes.cpu().numpy()
        at = np.nonzero(kept)
        assert np.array_equal(got[at[0], :, at[1]], c.codes[at[0], :, at[1]])
        assert np.array_equal(got[untouched], c.codes[untouched])


LAYOUTS = [
    (2, 64, [(200, 1)]),                                      # one new token
    (2, 64, [(16, 1), (17, 1), (1, 1), (32, 2)]),             # first and last slot, a block just begun
    (8, 128, [(100, 3), (33, 5), (48, 20), (7, 7), (64, 40)]),
    (3, 128, [(700, 700), (5, 5), (131, 90)]),                # prompts
    (40, 128, [(50, 1)] * 9),
    (1, 64, [(16, 16)] * 30 + [(15, 2)]),
]


@pytest.mark.parametrize("hkv,d,reqs", LAYOUTS)
def test_append(hkv, d, reqs):
    rng = np.random.default_rng(hkv * 100 + len(reqs))
    ctx = [c for c, _ in reqs]
    nb = sum((c + 15) // 16 for c in ctx) + 5
    pool = filled(nb, hkv, d, 3)
    bt = ref.tables(rng, ctx, nb)
    cu = np.cumsum([0] + [n for _, n in reqs])
    pos = np.concatenate([np.arange(c - n, c) for c, n in reqs])
    held = [c - n for c, n in reqs]
    k, v = rows(rng, (len(pos), hkv, d)), rows(rng, (len(pos), hkv, d))
    want = caches(pool)
    kept = [w.append(bt, cu, pos, held, x.double().numpy()) for w, x in zip(want, (k, v))][0]
    written = np.unique([bt[r][p // 16] for r in range(len(reqs)) for p in pos[cu[r]:cu[r + 1]]])
    run(pool, bt, cu, pos, held, k, v)
    check(pool, want, kept, np.setdiff1d(np.arange(nb), written))
    assert pkv.pkv_check_device_errors(pool) == 0


def test_a_token_at_a_time():
    """Blocks that grow: the exponent follows the largest row so far, held codes are rounded whenever it rises."""
    rng = np.random.default_rng(8)
    pool = filled(6, 2, 64, 4)
    bt = np.array([[3, 0], [5, -1]], np.int32)
    want = caches(pool)
    for p in range(20):
        live = [r for r in range(2) if p < (20, 9)[r]]
        pos, held = [p] * len(live), [p] * 2
        cu = np.cumsum([0] + [int(r in live) for r in range(2)])
        k, v = rows(rng, (len(live), 2, 64), 2.0), rows(rng, (len(live), 2, 64), 2.0)
        for w, x in zip(want, (k, v)):
            kept = w.append(bt, cu, pos, held, x.double().numpy())
        run(pool, bt, cu, pos, held, k, v)
        check(pool, want, kept, np.array([1, 2, 4]))


@pytest.mark.parametrize("held", [0, 5, 16, 40])
def test_rewritten_positions(held):
    """Positions below held_lens: written ones are replaced, the others of their blocks are kept."""
    rng = np.random.default_rng(held)
    pool = filled(4, 2, 128, 5)
    bt = np.array([[2, 0, 1]], np.int32)
    pos = [0, 1, 2, 18, 19, 31, 33]
    k, v = rows(rng, (7, 2, 128)), rows(rng, (7, 2, 128))
    want = caches(pool)
    kept = [w.append(bt, [0, 7], pos, [held], x.double().numpy()) for w, x in zip(want, (k, v))][0]
    run(pool, bt, [0, 7], pos, [held], k, v)
    check(pool, want, kept, np.array([3]))


def test_one_position_twice_and_any_order_within_a_block():
    rng = np.random.default_rng(77)
    pool = filled(3, 1, 64, 6)
    bt = np.array([[1, 2]], np.int32)
    pos = [7, 3, 7, 0] + [12] * 40 + [17, 16, 17]
    k, v = rows(rng, (len(pos), 1, 64)), rows(rng, (len(pos), 1, 64))
    want = caches(pool)
    kept = [w.append(bt, [0, len(pos)], pos, [2], x.double().numpy()) for w, x in zip(want, (k, v))][0]
    run(pool, bt, [0, len(pos)], pos, [2], k, v)
    check(pool, want, kept, np.array([0]))


@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -126, 2.0 ** -119, 1.0, 2.0 ** 120])
def test_range_of_values(scale):
    """Subnormals, the borders 127 * 2^e and 127.5 * 2^e, the largest bf16, held codes far below the new rows."""
    rng = np.random.default_rng(1)
    x = torch.zeros((6, 2, 64), dtype=torch.float64)
    x[0] = torch.tensor(rng.standard_normal((2, 64)))
    x[1, 0, 5], x[1, 1, 9] = 127.0 / 128, -127.5 / 128
    x[2, :, 0] = 254.0 / 256
    x[3, 0] = 255.0 / 256
    x[4, 1, 63] = -1.0
    x = (x * scale).clamp(-3.3895e38, 3.3895e38).to(torch.bfloat16)
    x[5] = 0
    if scale > 1:
        x[5, 0, 1] = 3.3895e38
    for order in ([0, 1, 2, 3, 4, 5], [5, 3, 0, 4, 2, 1]):
        pool = filled(2, 2, 64, 9)
        pool.k_exps.fill_(-126)
        want = caches(pool)
        for i, row in enumerate(order):
            one = x[row:row + 1]
            for w in want:
                kept = w.append([[1]], [0, 1], [i], [i], one.double().numpy())
            run(pool, np.array([[1]], np.int32), [0, 1], [i], [i], one, one)
            check(pool, want, kept, np.array([0]))
        k, v = pkv.pkv_read_rows(pool, ref.dev(np.array([[1]], np.int32)), ref.dev(np.array([0, 6], np.int32)),
                                 ref.dev(np.arange(6, dtype=np.int32)))
        assert torch.isfinite(k.float()).all()
        assert np.array_equal(k.cpu().double().numpy(), want[0].values()[1].transpose(1, 0, 2)[:6])
        assert np.array_equal(v.cpu().double().numpy(), want[1].values()[1].transpose(1, 0, 2)[:6])


def test_values_that_are_not_finite():
    rng = np.random.default_rng(2)
    k, v = rows(rng, (3, 2, 128)), rows(rng, (3, 2, 128))
    k[0, 0, 3] = float("inf")
    k[1, 1, 7] = float("nan")
    v[2, 0, 0] = float("-inf")
    v[2, 1, 1] = float("nan")
    pool = filled(2, 2, 128, 1)
    want = caches(pool)
    bt = np.array([[1]], np.int32)
    kept = [w.append(bt, [0, 3], [4, 5, 6], [4], x.double().numpy()) for w, x in zip(want, (k, v))][0]
    run(pool, bt, [0, 3], [4, 5, 6], [4], k, v)
    check(pool, want, kept, np.array([0]))
    assert pkv.pkv_check_device_errors(pool) == pkv.PKV_DEVERR_VALUE


def test_bad_slots_and_padding():
    """A position outside the table, a block id outside the pool, tokens behind the last request: the rest is written."""
    rng = np.random.default_rng(12)
    hkv, d = 2, 64
    k, v = rows(rng, (9, hkv, d)), rows(rng, (9, hkv, d))
    pool = filled(5, hkv, d, 2)
    want = caches(pool)
    bt = np.array([[3, 99], [-1, 4]], np.int32)
    cu, pos = [0, 4, 6], [0, 1, 17, 40, 3, 16, 0, 1, 2]
    good = np.array([[3, 99], [0, 4]])
    for w, x in zip(want, (k, v)):
        w.append(good[:1], [0, 2], pos[:2], [0], x[:2].double().numpy())
        kept = w.append(good[1:], [0, 1], [16], [16], x[5:6].double().numpy())
        kept[3, :2] = True
    run(pool, bt, cu, pos, [0, 16], k, v)
    check(pool, want, kept, np.array([0, 1, 2]))
    assert pkv.pkv_check_device_errors(pool) == pkv.PKV_DEVERR_BLOCK_ID | pkv.PKV_DEVERR_POSITION
    run(pool, bt[:, :1], [0, 2, 12], [0, 1], [2, 2], k[:2], v[:2])      # a range beyond the tokens
    assert pkv.pkv_check_device_errors(pool) & pkv.PKV_DEVERR_POSITION


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (40, 64)])
def test_read_rows(dtype, hkv, d):
    rng = np.random.default_rng(hkv + d)
    nb = 30
    if dtype == "int8":
        pool = filled(nb, hkv, d, 1)
        want = [c.values() for c in caches(pool)]
    else:
        pool = ref.random_pool(pkv.Pool(nb, hkv, d, dtype=dtype, k_scale=0.017 if dtype != "bf16" else 1.0, v_scale=0.5), 1)
        vals = [(x.cpu().view(torch.float8_e4m3fn) if dtype != "bf16" else x.cpu()).float() for x in (pool.k, pool.v)]
        want = [(x * torch.tensor(s if dtype != "bf16" else 1.0, dtype=torch.float32)).to(torch.bfloat16).double().numpy()
                for x, s in zip(vals, (pool.k_scale, pool.v_scale))]     # the product in fp32, rounded once more
    bt = ref.tables(rng, [200, 16, 100], nb)
    pos = np.concatenate([rng.integers(0, 200, 37), [0, 15, 15], rng.integers(0, 100, 5), [77, 78]]).astype(np.int32)
    cu = np.array([0, 37, 40, 45], np.int32)        # two rows that belong to no request
    out = [torch.full((len(pos), hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = pkv.pkv_read_rows(pool, ref.dev(bt), ref.dev(cu), ref.dev(pos), k_out=out[0], v_out=out[1])
    assert k is out[0] and v is out[1]
    req = np.repeat(np.arange(3), np.diff(cu))
    ids = bt[req, pos[:45] // 16]
    for got, w in zip((k, v), want):
        got = got.cpu().double().numpy()
        assert np.array_equal(got[:45], w[ids, :, pos[:45] % 16])
        assert (got[45:] == 7.0).all()
    assert pkv.pkv_check_device_errors(pool) == 0


def test_read_rows_that_are_not_there():
    pool = filled(3, 2, 64, 1)
    pos = np.array([0, 16, -1, 48, 33], np.int32)
    bt = np.array([[2, -1, 3]], np.int32)
    k, v = pkv.pkv_read_rows(pool, ref.dev(bt), ref.dev(np.array([0, 5], np.int32)), ref.dev(pos))
    assert torch.equal(k[0].float(), torch.ldexp(pool.k[2, :, 0].float(), pool.k_exps[2].int()[:, None]))
    assert (k[1:] == 0).all() and (v[1:] == 0).all()
    assert pkv.pkv_check_device_errors(pool) == pkv.PKV_DEVERR_BLOCK_ID | pkv.PKV_DEVERR_POSITION


def test_no_tokens():
    pool = filled(3, 2, 64, 1)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    bt, cu = ref.dev(np.zeros((1, 2), np.int32)), ref.dev(np.zeros(2, np.int32))
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_append_int8(pool, bt, cu, z, cu[:1], e, e)
    k, v = pkv.pkv_read_rows(pool, bt, cu, z)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)


def test_copies_and_forks_take_the_exponents_along():
    pool = filled(8, 3, 64, 1)
    pkv.pkv_copy_blocks(pool, ref.dev(np.array([0, 1], np.int32)), ref.dev(np.array([5, 2], np.int32)))
    for c, e in ((pool.k, pool.k_exps), (pool.v, pool.v_exps)):
        assert torch.equal(c[5], c[0]) and torch.equal(e[5], e[0]) and torch.equal(c[2], c[1]) and torch.equal(e[2], e[1])
    refs = ref.dev(np.array([1, 1, 0, 0, 0, 0, 0, 0], np.int32))
    i = lambda *x: ref.dev(np.array(x, np.int32))
    new, refs = pkv.pkv_fork(pool, i(0, 1).view(1, 2), i(20), i(20), i(0, 0), i(21, 21), refs)
    new = new.cpu().tolist()
    assert new[0] == [0, 1] and new[1][0] == 0 and new[1][1] not in (0, 1)
    pos = i(*range(20))
    for x in pkv.pkv_read_rows(pool, ref.dev(np.array(new, np.int32)), i(0, 20, 40), torch.cat([pos, pos])):
        assert torch.equal(x[:20], x[20:])


def test_streams_graphs_and_following_calls():
    """The write and the read captured together, replayed with other rows, lengths and tables."""
    rng = np.random.default_rng(3)
    pool = filled(12, 2, 128, 1)
    bt = ref.dev(ref.tables(rng, [60, 60], 12))
    cu, pos, held = ref.dev(np.array([0, 2, 4], np.int32)), ref.dev(np.array([3, 4, 30, 31], np.int32)), ref.dev(np.array([3, 30], np.int32))
    k, v = rows(rng, (4, 2, 128)).cuda(), rows(rng, (4, 2, 128)).cuda()
    out = [torch.empty_like(k), torch.empty_like(v)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkv.pkv_append_int8(pool, bt, cu, pos, held, k, v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkv.pkv_append_int8(pool, bt, cu, pos, held, k, v)
            pkv.pkv_read_rows(pool, bt, cu, pos, k_out=out[0], v_out=out[1])
        torch.cuda.synchronize()
        for step in range(3):
            k.copy_(rows(rng, (4, 2, 128)))
            v.copy_(rows(rng, (4, 2, 128)))
            pos.copy_(ref.dev(np.array([5 + 2 * step, 6 + 2 * step, 32 + 2 * step, 33 + 2 * step], np.int32)))
            held.copy_(ref.dev(np.array([5 + 2 * step, 32 + 2 * step], np.int32)))
            torch.cuda.synchronize()
            want = caches(pool)
            h, p, b = held.cpu().numpy(), pos.cpu().numpy(), bt.cpu().numpy()
            for w, x in zip(want, (k, v)):
                kept = w.append(b, [0, 2, 4], p, h, x.cpu().double().numpy())
            g.replay()
            check(pool, want, kept, np.array([], np.int64))
            ids = b[[0, 0, 1, 1], p // 16]
            for x, w in zip(out, want):
                assert np.array_equal(x.cpu().double().numpy(), w.values()[ids, :, p % 16])


def test_refusals():
    pool = filled(3, 2, 64, 1)
    bf = pkv.Pool(3, 2, 64)
    i = lambda *x: ref.dev(np.array(x, np.int32))
    bt, cu, pos = i(0).view(1, 1), i(0, 1), i(0)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_append_int8(bf, bt, cu, pos, pos, x, x)
    assert e.value.code == pkv.PKV_EINVAL
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    meta = pkv.HostMeta([0, 1], [1], [0])
    buf = torch.zeros(2 * 2 * 16 * 64, dtype=torch.uint8).pin_memory()
    z = torch.zeros((3, 2, 2, 64), dtype=torch.int8, device="cuda"), torch.zeros((3, 2), dtype=torch.int8, device="cuda")
    summary = pkv.BlockSummary(pool, *z)
    mask = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: pkv.pkv_append(pool, bt, cu, pos, x, x),
                 lambda: pkv.pkv_paged_attn(pool, q, pos, bt, i(1), cu, meta, 1.0),
                 lambda: pkv.pkv_append_paged_attn(pool, q, pos, bt, i(1), cu, meta, x, x, 1.0),
                 lambda: pkv.pkv_paged_attn_static(pool, q, pos, bt, i(1), cu, meta, 1.0),
                 lambda: pkv.pkv_tree_attn(pool, q, bt, i(1), i(0), cu, mask, 1.0),
                 lambda: pkv.pkv_summarize(pool, summary, bt, cu, pos, i(1)),
                 lambda: pkv.pkv_select_blocks(pool, summary, q, pos, bt, cu, 1),
                 lambda: pkv.pkv_sparse_attn(pool, q, pos, bt, cu, i(0, 0).view(1, 2, 1), 1.0),
                 lambda: pkv.pkv_compact(pool, bt, cu, pos, pos),
                 lambda: pkv.pkv_swap_out(pool, np.array([0]), buf),
                 lambda: pkv.pkv_swap_in(pool, np.array([0]), buf),
                 lambda: pkv.pkv_swap_in_ahead(pool, np.array([0]), buf, torch.cuda.Stream())):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.code == pkv.PKV_EUNSUPPORTED
    with pytest.raises(TypeError):
        pkv.pkv_append_int8(pool, bt, cu, pos, pos, x.float(), x)
    with pytest.raises(ValueError):
        pkv.pkv_append_int8(pool, bt, cu, pos, i(0, 0), x, x)
    with pytest.raises(ValueError):
        pkv.pkv_read_rows(pool, bt, cu, pos, k_out=x[:, :1].contiguous())
    with pytest.raises(ValueError):
        pkv.Pool(3, 2, 64, dtype="int8", k_exps=pool.k_exps, v_exps=pool.v_exps)
    with pytest.raises(ValueError):
        pkv.Pool(3, 2, 64, k_exps=pool.k_exps, v_exps=pool.v_exps)
