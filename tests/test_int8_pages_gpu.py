"""The 8-bit cache in the steps of a block manager: leading blocks recomputed on pages that others left."""
import numpy as np
import pytest

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv
from test_int8_gpu import built, caches, check, filled, rows, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left", [-126, 100])
def test_blocks_that_are_written_whole_keep_nothing(left, d):
    """A conversation of 37 tokens whose first two blocks were dropped: the step recomputes them on fresh pages and adds two
    tokens, held_lens being the old length.  The exponents that earlier owners left on the pages have no say, the third
    block's, which keeps its five tokens, has."""
    rng = np.random.default_rng(left + 200)
    pool = filled(6, 3, d, 21)
    bt = np.array([[4, 1, 2]], np.int32)
    for e in (pool.k_exps, pool.v_exps):
        e[[4, 1]] = left
    pos = list(range(32)) + [37, 38]
    k, v = rows(rng, (34, 3, d)), rows(rng, (34, 3, d))
    want = caches(pool)
    for w, x in zip(want, (k, v)):
        x = x.double().numpy()
        kept = w.append(bt, [0, 32], pos[:32], [0], x[:32])
        kept |= w.append(bt, [0, 2], pos[32:], [37], x[32:])
    run(pool, bt, [0, 34], pos, [37], k, v)
    check(pool, want, kept, np.array([0, 3, 5]))
    assert pkv.pkv_check_device_errors(pool) == 0


def test_a_rewritten_slot_leaves_its_block_to_the_others():
    """One of two held slots written anew: the other keeps its value, and with it the block's exponent.  Both: it goes."""
    rng = np.random.default_rng(22)
    for pos, stays in (([1, 5], True), ([5, 0], True), ([1, 0], False), ([0, 1, 2, 0], False)):
        pool = filled(2, 2, 64, 23)
        pool.k_exps.fill_(3)
        pool.v_exps.fill_(3)
        k, v = rows(rng, (len(pos), 2, 64)), rows(rng, (len(pos), 2, 64))
        want = caches(pool)
        kept = [w.append([[1]], [0, len(pos)], pos, [2 if stays else 0], x.double().numpy()) for w, x in zip(want, (k, v))][0]
        run(pool, np.array([[1]], np.int32), [0, len(pos)], pos, [2], k, v)
        check(pool, want, kept, np.array([0]))


def test_a_manager_without_a_host_tier_drops_and_recomputes():
    """pkv_cache_step over an int8 pool (cpu_blocks = 0: nothing is swapped): every conversation's cache holds its rows to half
    a step of the exponent that fits the block."""
    rng = np.random.default_rng(24)
    hkv, d, blocks = 2, 64, 8
    pool = pkv.Pool(blocks, hkv, d, dtype="int8")
    cache = pkv.Cache(blocks, 0)
    text = {c: rows(rng, (100, hkv, d), 1.5) * 2.0 ** (6 * c - 6) for c in range(3)}      # of very different sizes
    length = {c: 0 for c in range(3)}
    recomputed = 0
    for c, n in ((0, 40), (1, 50), (2, 30), (0, 9), (1, 1), (2, 35), (0, 3), (1, 6)):
        step = cache.step([c], [n], 8)
        old, now, again = length[c], int(step["ctx_lens"][0]), int(step["recompute"][0])
        assert len(step["swap_out"]) == len(step["swap_in"]) == 0
        recomputed += again
        pos = list(range(min(again, old))) + list(range(old, now))
        x = text[c][pos]
        run(pool, step["block_tables"], [0, len(pos)], pos, [old], x, x)
        length[c] = now
        k, v = pkv.pkv_read_rows(pool, ref.dev(step["block_tables"]), ref.dev(np.array([0, now], np.int32)),
                                 ref.dev(np.arange(now, dtype=np.int32)))
        src = text[c][:now].double().numpy()
        for got in (k, v):
            err = np.abs(got.double().cpu().numpy() - src)
            for b in range(0, now, 16):
                # Half a step when written, half of the new one each time the exponent grows: 2^e in all at most, the steps
                # being powers of two, and 127 * 2^e is less than twice the block's largest value.
                top = np.abs(src[b:b + 16]).max(axis=(0, 2))
                assert (err[b:b + 16].max(axis=(0, 2)) <= 2 * top / 127).all()
    assert recomputed > 0
    assert pkv.pkv_check_device_errors(pool) == 0
