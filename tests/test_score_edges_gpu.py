"""Attention with modified scores at the edges of what its documentation allows: tables with invalid ids where nobody looks,
tokens that see nothing, the corners of the cap's range, batches of more requests and items than the plan keeps at hand."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import score_ref
from paged_kv_attention_25_gb300 import pkv
from test_score_gpu import DTYPES, Case, built, make_pool, tail, values  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
TYPES = pytest.mark.parametrize("dtype", DTYPES)


def forced(case, form):
    pkv.pkv_debug_set(case.pool, pkv.PKV_DEBUG_TREE_FORM, form)
    return case


def unseen_blocks(c):
    """(request, block) pairs of the table of which no token of the request sees a key, beyond the context among them."""
    out = []
    for r in range(len(c.ctx)):
        ctx = int(c.ctx[r])
        seen = np.zeros(c.bt.shape[1] * 16, bool)
        for t in range(c.cu[r], c.cu[r + 1]):
            seen[:ctx] |= score_ref.sees(int(c.pos[t]), ctx, 0 if c.prefix is None else int(c.prefix[r]),
                                         0 if c.first is None else int(c.first[t]), c.window)
        out += [(r, b) for b in np.nonzero(~seen.reshape(-1, 16).any(1))[0]]
    return out


def check_unseen_ids(c, inside):
    """Bad ids in the blocks that nobody sees, `inside` of them within the contexts at least, change nothing and are no error."""
    want = c.call()
    c.check(*want)
    assert pkv.pkv_check_device_errors(c.pool) == 0
    gone = unseen_blocks(c)
    assert sum(b * 16 < c.ctx[r] for r, b in gone) >= inside
    for i, (r, b) in enumerate(gone):
        c.bt[r, b] = (-1, c.pool.num_blocks, -2 ** 31, 2 ** 31 - 1)[i % 4]
    got = c.call()
    assert pkv.pkv_check_device_errors(c.pool) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


UNSEEN = {
    # windows that begin anywhere in a tile of 128 keys, with and without a few leading tokens
    "window": ([tail(700, 3), tail(391, 9), tail(200, 1), tail(129, 2)], dict(window=100), 60),
    "window_prefix": ([tail(700, 3), tail(391, 9), tail(200, 1)], dict(window=45, prefix=[5, 17, 0]), 60),
    "window_cap_slopes": ([tail(523, 40), tail(260, 2)], dict(window=33, softcap=4.0, slopes=True), 40),
    # positions well below the contexts' ends
    "behind": ([(400, [100, 101, 102, 103]), (300, [0]), (150, list(range(20, 60)))], {}, 35),
    # prompts of several tiles whose first tokens have left the window of the last
    "prompts": ([tail(1500, 300), tail(900, 150)], dict(window=70), 100),
}


@FORMS
@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", list(UNSEEN))
def test_block_ids_that_nobody_sees_are_not_looked_at(what, d, dtype, form):
    reqs, opts, inside = UNSEEN[what]
    check_unseen_ids(forced(Case(100, reqs, 8, 2, d, dtype, **opts), form), inside)


@FORMS
@TYPES
def test_block_ids_before_a_document(dtype, form):
    c = forced(Case(101, [tail(600, 50), tail(333, 3)], 8, 2, 64, dtype), form)
    c.first = np.concatenate([np.full(50, 505), np.full(3, 300)]).astype(np.int32)
    check_unseen_ids(c, 45)


@FORMS
@pytest.mark.parametrize("scale,softcap", [(2.0 ** 44, 2.0 ** 29), (2.0 ** 10, 2.0 ** -9), (2.0 ** -40, 2.0 ** -18), (2.0 ** 30, 2.0 ** 30)])
def test_caps_and_scales_far_from_one(scale, softcap, form):
    """Queries as small as the scale is large (and the reverse), so that scores lie on both sides of half the cap, where that
    is anything: products of powers of two, exact in every step before the cap."""
    c = forced(Case(110, [tail(200, 20)], 4, 2, 64, scale=scale, softcap=softcap), form)
    size = min(softcap, 8.0) / scale / 8
    c.q = (c.q.float() * 2.0 ** round(np.log2(size))).to(torch.bfloat16)
    o, lse = c.call()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    if softcap >= 2.0 ** 20:      # scores below 2^-17 of the cap: the formula without it is off by 2^-35 of them, and its bounds
        c.cap = 0.0               # hold, as the polynomial's 6e-7 of a score below 32 is less than their 2^-15
    c.check(o, lse)
    c.q = torch.zeros_like(c.q)
    c.check(*c.call())
    assert pkv.pkv_check_device_errors(c.pool) == 0


@FORMS
def test_scales_whose_products_leave_fp32_are_refused(form):
    """scale, scale * k_scale or their quotient by softcap, as the scores are made with them, have to be normal numbers."""
    f32 = lambda x: float(np.float32(x))
    ok = [("bf16", 2.0 ** 126, 0.0, 1.0), ("fp8_e4m3", 2.0 ** 96, 0.0, 2.0 ** 30), ("fp8_e4m3", 2.0 ** -63, 0.0, 2.0 ** -63),
          ("bf16", 2.0 ** 97, 2.0 ** -30, 1.0), ("bf16", 2.0 ** -96, 2.0 ** 30, 1.0)]
    bad = [("bf16", f32(3e38), 0.0, 1.0), ("fp8_e4m3", 2.0 ** 98, 0.0, 2.0 ** 30), ("bf16", 2.0 ** 98, 2.0 ** -30, 1.0),
           ("bf16", 2.0 ** -97, 2.0 ** 30, 1.0), ("fp8_e4m3", 2.0 ** -40, 2.0, 2.0 ** -100), ("int8", f32(3e38), 0.0, 1.0),
           ("fp8_e4m3", f32(1e-30), 0.0, f32(1e-30)), ("bf16", 2.0 ** -128, 0.0, 1.0)]
    for i, (dtype, scale, softcap, k_scale) in enumerate(ok + bad):
        c = Case(120, [tail(20, 2)], 4, 2, 64, dtype, scale=scale, softcap=softcap)
        if dtype == "fp8_e4m3":
            c.pool = pkv.Pool(c.pool.num_blocks, 2, 64, dtype=dtype, k_scale=k_scale, v_scale=0.5)
        forced(c, form)
        c.q = torch.zeros_like(c.q)          # (scores of zero whatever the scale)
        if i < len(ok):
            c.check(*c.call())
            continue
        with pytest.raises(pkv.PkvError) as e:
            c.call()
        assert e.value.code == pkv.PKV_EINVAL


@FORMS
def test_int8_keys_of_the_largest_exponent(form):
    """Products that are zero give scores of zero whatever the exponent and the scale; those that are not are fp32 numbers."""
    c = forced(Case(121, [tail(80, 3), tail(33, 1)], 4, 2, 64, "int8", scale=200.0), form)
    c.pool.k_exps.fill_(121)
    c.q = torch.zeros_like(c.q)
    c.q[1, 2, 5] = 2.0 ** -120
    c.check(*c.call())
    assert pkv.pkv_check_device_errors(c.pool) == 0


@FORMS
@TYPES
def test_tokens_that_see_nothing_do_not_widen_what_is_read(dtype, form):
    """A document that begins behind its token, a token in front of the sequence: the blocks between are still nobody's."""
    c = forced(Case(122, [(700, [20, 690, 21, 691]), (512, [100, 500])], 8, 2, 64, dtype, window=30), form)
    c.first = np.array([300, 600, 22, 0, 400, 0], np.int32)
    c.pos[2] = 21
    check_unseen_ids(c, 60)
    c = forced(Case(123, [(700, [3, 690, 691])], 8, 2, 64, dtype, window=30, prefix=[7]), form)
    c.pos[0] = -5
    for r, b in unseen_blocks(c):
        c.bt[r, b] = -1
    c.check(*c.call())
    assert pkv.pkv_check_device_errors(c.pool) == pkv.PKV_DEVERR_POSITION


def test_token_ranges_that_overlap_beyond_32_bits():
    """Half of 180 thousand requests claim all of 100 thousand tokens each: 4.5e9 pairs of tiles, cut to what the plan has
    room for and flagged.  All requests have the same page, so that whoever writes a row writes the same."""
    tokens, reqs, hq, d = 100_000, 180_000, 128, 64
    pool = make_pool(3, 1, d, "bf16", 130)
    pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, 2)
    q = torch.randn((tokens, hq, d), generator=torch.Generator("cuda").manual_seed(131), device="cuda").to(torch.bfloat16)
    i32 = lambda n, x: torch.full((n,), x, dtype=torch.int32, device="cuda")
    cu = i32(reqs + 1, 0)
    cu[1::2] = tokens
    o, lse = pkv.pkv_score_attn(pool, q, i32(tokens, 5), i32(reqs, 1).view(-1, 1), i32(reqs, 16), cu, 0.125)
    assert pkv.pkv_check_device_errors(pool) == pkv.PKV_DEVERR_POSITION
    k, v = (values(pool, w)[1, 0] for w in "kv")
    for t in (0, 1, 49_999, 77_776, tokens - 1):
        want, wl, tol, tl = score_ref.rows(q[t].double().cpu().numpy(), k, v, 5, np.arange(16) <= 5, 0.125, 0.0, None, False)
        ref.assert_close(o[t].double().cpu().numpy(), want, tol, f"O of token {t}")
        ref.assert_close(lse[t].double().cpu().numpy(), wl, tl, f"LSE of token {t}")


@TYPES
@pytest.mark.parametrize("reqs,toks,hq", [(1100, 1, 8), (5, 900, 128), (1500, 3, 128)],
                         ids=["many_requests", "many_items", "both"])
def test_plans_beyond_what_is_kept_at_hand(reqs, toks, hq, dtype):
    """More than 1,024 requests, more than 2,048 items of two tiles (tiles of one token with 128 rows), and both."""
    rng = np.random.default_rng(132)
    ctxs = rng.integers(toks, toks + 40, reqs)
    c = forced(Case(133, [tail(int(x), toks) for x in ctxs], hq, 1, 64, dtype, extra=2, window=30, softcap=6.0), 2)
    o, lse = c.call()
    last = len(c.pos) - 3
    c.check(o, lse, {0, 1, 2, last // 2, last - 1, last} | set(rng.integers(0, last, 40).tolist()))
    assert torch.isfinite(o[:last + 1]).all() and torch.isfinite(lse[:last + 1]).all()
    assert pkv.pkv_check_device_errors(c.pool) == 0
    # Every request and tile is served: as in the rows form.  Each is off by 2^-8 A for P and 2^-8 |O| for O, A and |O| at
    # most the largest |v|, and by half as much again for everything else.
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_TREE_FORM, 1)
    p, m = c.call()
    most = np.abs(values(c.pool, "v")).max()
    assert (o[:last + 1].float() - p[:last + 1].float()).abs().max() <= 2 * 2.5 * 2.0 ** -8 * most
    assert (lse[:last + 1] - m[:last + 1]).abs().max() <= 1e-3


@TYPES
@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
def test_rows_without_a_key_in_every_type(dtype, form):
    """(And documents that leave some tokens nothing, and requests without a context.)"""
    c = forced(Case(134, [tail(40, 3), tail(300, 7), tail(16, 2), (0, []), tail(129, 5), tail(2, 2)], 8, 2, 128, dtype, docs=5), form)
    c.run()
    assert c.seen_empty


@TYPES
@pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])
def test_scores_beyond_the_cap_in_every_type(dtype, form):
    reqs = [tail(50, 50), tail(200, 3)]
    forced(Case(135, reqs, 8, 2, 64, dtype, softcap=30.0, scale=40.0), form).run()
    forced(Case(136, reqs, 8, 2, 128, dtype, softcap=5.0, slopes=True, scale=3.0), form).run()
    c = forced(Case(137, reqs, 4, 2, 64, dtype, slopes=True), form)
    c.slopes = np.array([100.0, -0.25, 0.0, 1e-3], np.float32)
    c.run()


@FORMS
def test_exponents_outside_their_range_are_read_as_the_nearest(form):
    """Pages that the table names, with exponents that no append writes.  K: large ones, under queries small enough; V: one page
    of large ones (codes of at most 1: 16 of them stay in fp32's range), then small ones alone, and zeros under any."""
    c = forced(Case(140, [tail(90, 4), tail(33, 2)], 4, 2, 64, "int8"), form)
    gen = torch.Generator("cuda").manual_seed(141)
    sign = torch.where(torch.rand(c.q.shape) < 0.5, -1.0, 1.0)
    big, tiny, zero = (c.bt[0][1], c.bt[1][0]), (c.bt[0][0], c.bt[1][1]), c.bt[0][3]
    for i, e in zip(big, (127, 122)):
        c.pool.k[i] = torch.randint(-3, 4, c.pool.k[i].shape, generator=gen, device="cuda")
        c.pool.k_exps[i] = e
    for i, e in zip(tiny, (-128, -127)):
        c.pool.k_exps[i] = e
    c.pool.k[zero], c.pool.k_exps[zero] = 0, 127
    c.q = (sign * (0.5 + torch.rand(c.q.shape))).mul(2.0 ** -119).to(torch.bfloat16)
    c.check(*c.call())
    c.q = (sign * torch.rand(c.q.shape)).to(torch.bfloat16)
    for i in big:
        c.pool.k_exps[i] = -7
    c.pool.v[big[0]] = torch.randint(-1, 2, c.pool.v[big[0]].shape, generator=gen, device="cuda")
    c.pool.v_exps[big[0]] = 127
    c.pool.v[zero], c.pool.v_exps[zero] = 0, 122
    c.check(*c.call())
    assert pkv.pkv_check_device_errors(c.pool) == 0


@FORMS
def test_int8_values_below_bf16s_weights(form):
    """Exponents of -126 and below everywhere.  The rows form's weights times 2^e (times 2^6, the widening's) are bf16
    numbers below its normal ones: each is off by 2^-134 at most, times a code of 127 / 64 at most, 2^-133 a key; O is
    off by 2^-134 where it has no normal bf16 number."""
    c = forced(Case(142, [tail(150, 4), tail(33, 2), tail(600, 1)], 8, 2, 64, "int8"), form)
    for e in (-126, -128):
        c.pool.v_exps.fill_(e)
        o, lse = c.call()
        o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
        k, v, q = values(c.pool, "k"), values(c.pool, "v"), c.q.double().numpy()
        for r in range(3):
            ctx = int(c.ctx[r])
            for g in range(2):
                kk, vv = (ref.gather(x, c.bt[r], ctx, g)[0] for x in (k, v))
                hs = slice(4 * g, 4 * g + 4)
                for t in range(c.cu[r], c.cu[r + 1]):
                    seen = np.arange(ctx) <= c.pos[t]
                    want, wl, tol, tl = score_ref.rows(q[t, hs], kk, vv, int(c.pos[t]), seen, c.scale, 0.0, None, False)
                    ref.assert_close(o[t, hs], want, tol + seen.sum() * 2.0 ** -133 + 2.0 ** -134, f"O of token {t}")
                    ref.assert_close(lse[t, hs], wl, tl, f"LSE of token {t}")


@pytest.mark.parametrize("d", [64, 128])
def test_rows_read_back_with_exponents_outside_their_range(d):
    pool = make_pool(5, 3, d, "int8", 143)
    exps = [-128, -127, -126, 121, 122]
    for i, e in enumerate(exps):
        pool.k_exps[i], pool.v_exps[i] = e, (127 if e == 122 else e)
    pos = np.arange(80, dtype=np.int32)
    k, v = pkv.pkv_read_rows(pool, ref.dev(np.arange(5, dtype=np.int32)[None]), ref.dev(np.array([0, 80], np.int32)), ref.dev(pos))
    for got, which in ((k, "k"), (v, "v")):
        want = values(pool, which).transpose(0, 2, 1, 3).reshape(80, 3, d)
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert pkv.pkv_check_device_errors(pool) == 0


@FORMS
@TYPES
def test_tokens_inside_the_prefix_do_not_widen_what_is_read(dtype, form):
    """A window or document that lies inside the prefix adds nothing to it, and no blocks between it and the others' keys."""
    c = forced(Case(124, [(900, [200, 880, 299, 881]), (700, [690, 30]), (400, [150, 100])], 8, 2, 64, dtype, window=30,
                    prefix=[300, 45, 200]), form)
    check_unseen_ids(c, 70)
