"""The 8-bit cache's calls and the attention with modified scores in the order in which they are issued: behind swap-ins that
are under way, right behind writes, with launches counted."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from paged_kv_attention_25_gb300 import pkv
from test_int8_gpu import rows
from test_score_gpu import DTYPES, Case, built, make_pool, tail, values  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = pytest.mark.parametrize("form", [1, 2], ids=["rows", "tiles"])


@FORMS
@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("call", ["attend", "read"])
def test_a_swap_in_that_is_under_way_lands_first(call, dtype, form):
    c = Case(200, [tail(150, 3), tail(70, 20)], 8, 2, 64, dtype, softcap=5.0)
    pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_TREE_FORM, form)
    bt, cu, pos, ctx, q = ref.dev(c.bt), ref.dev(c.cu), ref.dev(c.pos), ref.dev(c.ctx), c.q.cuda()
    if call == "attend":
        go = lambda: pkv.pkv_score_attn(c.pool, q, pos, bt, ctx, cu, c.scale, softcap=5.0)
    else:
        go = lambda: pkv.pkv_read_rows(c.pool, bt, cu, pos)
    want = go()
    ids = np.array([int(c.bt[0][2]), int(c.bt[0][9]), int(c.bt[1][4])], np.int32)
    host = torch.empty((3, 2, 2, 16, 64), dtype=c.pool.k.dtype).pin_memory()
    pkv.pkv_swap_out(c.pool, ids, host)
    torch.cuda.synchronize()
    c.pool.k[ids.tolist()] = 0
    c.pool.v[ids.tolist()] = 0
    pkv.pkv_swap_in_ahead(c.pool, ids, host, torch.cuda.Stream())
    got = go()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a call that is captured is refused while one is pending, and goes when it has landed
    pkv.pkv_swap_in_ahead(c.pool, ids, host, torch.cuda.Stream())
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with pytest.raises(pkv.PkvError) as e:
        with torch.cuda.graph(g, stream=s):
            go()
    assert e.value.code == pkv.PKV_EINVAL
    torch.cuda.synchronize()
    pkv.pkv_swap_in_finish(c.pool)
    got = go()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pkv.pkv_check_device_errors(c.pool) == 0


@FORMS
def test_steps_issued_without_waiting(form):
    """Append, attention and reading back, 60 steps of them queued at once, each step over what the last one wrote: the bits
    are those of the same steps with a wait behind every call."""
    rng = np.random.default_rng(201)
    ctx0, hkv, d = [300, 61, 16], 2, 128
    n, steps = [3, 1, 20], 60
    data = [(rows(rng, (24, hkv, d), 1.0).cuda(), rows(rng, (24, hkv, d), 1.0).cuda(), rows(rng, (24, 8, d), 0.5).cuda())
            for _ in range(steps)]
    lens = np.array(ctx0)[None] + np.arange(steps)[:, None] * np.array(n)
    bt = ref.dev(ref.tables(rng, (lens[-1] + n).tolist(), 200))
    meta = []
    for i in range(steps):
        pos = np.concatenate([np.arange(l, l + k) for l, k in zip(lens[i], n)]).astype(np.int32)
        meta.append((ref.dev(pos), ref.dev(lens[i].astype(np.int32)), ref.dev((lens[i] + n).astype(np.int32))))
    cu = ref.dev(np.cumsum([0] + n).astype(np.int32))
    outs = []
    for wait in (True, False):
        pool = make_pool(200, hkv, d, "int8", 202)
        pkv.pkv_debug_set(pool, pkv.PKV_DEBUG_TREE_FORM, form)
        got = []
        torch.cuda.synchronize()
        for (k, v, q), (pos, held, ctx) in zip(data, meta):
            for f in (lambda: pkv.pkv_append_int8(pool, bt, cu, pos, held, k, v),
                      lambda: pkv.pkv_score_attn(pool, q, pos, bt, ctx, cu, d ** -0.5, softcap=8.0, window=200),
                      lambda: pkv.pkv_read_rows(pool, bt, cu, pos)):
                x = f()
                if x is not None:
                    got += x
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append(got + [pool.k, pool.v, pool.k_exps, pool.v_exps])
        assert pkv.pkv_check_device_errors(pool) == 0
    assert len(outs[0]) == len(outs[1])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_launches_are_counted_where_the_header_says():
    c = Case(203, [tail(900, 40), tail(33, 1)], 8, 2, 64, "int8")
    pkv.pkv_profile_enable(c.pool, True)
    kinds = list(pkv.pkv_profile_read(c.pool, reset=True))
    new = rows(np.random.default_rng(204), (41, 2, 64), 1.0).cuda()
    held = ref.dev(c.ctx - np.diff(c.cu).astype(np.int32))
    counts = []
    for form in (1, 2):
        pkv.pkv_debug_set(c.pool, pkv.PKV_DEBUG_TREE_FORM, form)
        c.call()
        p = pkv.pkv_profile_read(c.pool, reset=True)
        counts.append([p[k]["launches"] for k in kinds])
        assert all(p[k]["total_ms"] > 0 for k in kinds if p[k]["launches"])
    pkv.pkv_append_int8(c.pool, ref.dev(c.bt), ref.dev(c.cu), ref.dev(c.pos), held, new, new)
    pkv.pkv_read_rows(c.pool, ref.dev(c.bt), ref.dev(c.cu), ref.dev(c.pos))
    p = pkv.pkv_profile_read(c.pool, reset=True)
    counts.append([p[k]["launches"] for k in kinds])
    assert counts[0][:3] == [0, 1, 0] and counts[1][:4] == [0, 0, 1, 1] and counts[2] == [2, 0, 0, 0, 0]
    pkv.pkv_profile_enable(c.pool, False)
