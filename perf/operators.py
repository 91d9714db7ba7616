"""What is measured of the cache operators beside the causal paged attention.

Three groups, each over the same block pool ([blocks][kv heads][16][head_dim], bf16 or e4m3 codes):

  tree       attention of drafted tokens over a cache: every token sees its request's prefix and the drafted
             slots that its bit mask names.
  sparse     attention over the blocks that a bound on the scores selects for each token ("summarize" builds
             the bounds, "sparse" selects and attends).
  pages      "fork" shares, copies, allocates and frees pages for the next generation of sequences; "compact"
             moves the rows of the drafted tokens that were kept to the front of the drafts.

`run` computes an operator in elementary torch operations, or (own = True) calls the library.
"""
import math
import random

import torch

own = False

BLOCK = 16
DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One conversation and a short drafted chain with two branches: what a single user's decode step costs.
        dict(name="tree_one_user", op="tree", reqs=1, ctx_lo=190, ctx_hi=240, nodes_lo=7, nodes_hi=7, hq=8, hkv=2, d=64,
             dtype="bf16", shape_seed=1),
        # A serving batch with grouped heads and trees of up to 64 nodes over ragged, partly long contexts: many rows
        # for each key, and keys that have to be split over the machine.
        dict(name="tree_batch_grouped", op="tree", reqs=12, ctx_lo=1500, ctx_hi=40000, nodes_lo=40, nodes_hi=64, hq=64,
             hkv=8, d=128, dtype="bf16", shape_seed=2),
        # Many heads with their own keys, small odd trees, 8-bit cache: bound by reading the cache.
        dict(name="tree_batch_fp8", op="tree", reqs=24, ctx_lo=300, ctx_hi=4000, nodes_lo=5, nodes_hi=27, hq=40, hkv=40,
             d=128, dtype="fp8_e4m3", shape_seed=3),
        # One conversation of a small model, one token: select 16 of about 190 blocks and attend to them.
        dict(name="sparse_one_user", op="sparse", reqs=1, ctx_lo=2900, ctx_hi=3100, toks_lo=1, toks_hi=1, hq=8, hkv=2, d=64,
             dtype="bf16", top_k=16, sinks=1, recent=2, shape_seed=5),
        # Decode of a batch of long contexts with grouped heads: an eighth of the cache is read.
        dict(name="sparse_batch_grouped", op="sparse", reqs=32, ctx_lo=9000, ctx_hi=40000, toks_lo=1, toks_hi=1, hq=64,
             hkv=8, d=128, dtype="bf16", top_k=128, sinks=1, recent=4, shape_seed=6),
        # Very long contexts with a key head for each query head and an 8-bit cache, one to three tokens a request.
        dict(name="sparse_long_fp8", op="sparse", reqs=5, ctx_lo=60000, ctx_hi=131000, toks_lo=1, toks_hi=3, hq=40, hkv=40,
             d=128, dtype="fp8_e4m3", top_k=64, sinks=2, recent=2, shape_seed=7),
        # The bounds after a decode step: the last block of each request.
        dict(name="summarize_step", op="summarize", reqs=64, ctx_lo=100, ctx_hi=400, toks_lo=1, toks_hi=2, hq=64, hkv=8,
             d=128, dtype="bf16", shape_seed=8),
        # The bounds of freshly prefilled prompts.
        dict(name="summarize_prompts", op="summarize", reqs=6, ctx_lo=3000, ctx_hi=9000, toks_lo=3000, toks_hi=9000, hq=64,
             hkv=8, d=128, dtype="bf16", shape_seed=9),
        # Four beams of one prompt move on by a token.
        dict(name="fork_beams", op="fork", groups=1, beams=4, ctx_lo=100, ctx_hi=140, hkv=2, d=64, room=1, shape_seed=10),
        # A batch of prompts with several samples each: some die, some are continued twice, all make room for drafts.
        dict(name="fork_batch", op="fork", groups=48, beams=5, ctx_lo=200, ctx_hi=2000, hkv=4, d=128, room=33,
             shape_seed=11),
        # The kept drafted tokens of one user's verified tree move to the front.
        dict(name="compact_one_user", op="compact", reqs=1, ctx_lo=200, ctx_hi=300, nodes_lo=16, nodes_hi=16, keep_hi=6,
             hkv=8, d=64, shape_seed=12),
        # The same for a large batch.
        dict(name="compact_batch", op="compact", reqs=128, ctx_lo=100, ctx_hi=700, nodes_lo=20, nodes_hi=64, keep_hi=14,
             hkv=8, d=128, shape_seed=13),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "sparse", "sparse", "sparse", "summarize", "fork", "fork", "compact"])
    hkv, group = rng.choice([(1, 8), (2, 1), (2, 4), (3, 5), (4, 2), (8, 1), (8, 8), (5, 1), (40, 1), (8, 4)])
    d = rng.choice([64, 128, 128])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=d, dtype=rng.choice(["bf16", "bf16", "fp8_e4m3"]),
             shape_seed=rng.randrange(1 << 30))
    if op in ("tree", "sparse", "summarize"):
        # Tokens of cache in the batch, times key heads, stay below the largest listed case.
        hi = _log_uniform(rng, 100, 60000)
        most = 700_000 // (hkv * hi)
        c["reqs"] = max(1, min(_log_uniform(rng, 1, 64), most))
        c["ctx_hi"] = max(64, min(hi, 700_000 // hkv))
        c["ctx_lo"] = max(40, c["ctx_hi"] // rng.choice([2, 8, 50]))
        if op == "tree":
            c["nodes_hi"] = min(_log_uniform(rng, 1, 64), max(1, 1024 // (group * 2)), c["ctx_lo"])
            c["nodes_lo"] = max(1, c["nodes_hi"] // rng.choice([1, 2, 5]))
        elif op == "summarize":
            c["toks_hi"] = _log_uniform(rng, 1, c["ctx_hi"])
            c["toks_lo"] = max(1, c["toks_hi"] // rng.choice([1, 3]))
        else:
            c["toks_hi"] = min(_log_uniform(rng, 1, 40), c["ctx_lo"])
            c["toks_lo"] = max(1, c["toks_hi"] // rng.choice([1, 3]))
            c["reqs"] = max(1, min(c["reqs"], 96 // c["toks_hi"]))
            c["top_k"] = max(4, min(_log_uniform(rng, 4, 128), 32768 // (c["reqs"] * c["toks_hi"] * hkv)))
            c["sinks"] = rng.choice([0, 1, 2])
            c["recent"] = rng.choice([1, 2, 3])
    elif op == "fork":
        c.update(groups=_log_uniform(rng, 1, 40), beams=rng.randint(1, 6), room=rng.choice([1, 1, 16, 17, 33]))
        c["ctx_hi"] = min(_log_uniform(rng, 40, 2000), 40 * 2000 // c["groups"])
        c["ctx_hi"] = max(40, c["ctx_hi"])
        c["ctx_lo"] = max(20, c["ctx_hi"] // rng.choice([2, 10]))
        c["hkv"] = min(hkv, 4)
        del c["dtype"], c["hq"]
    else:
        c.update(reqs=_log_uniform(rng, 1, 128), ctx_hi=_log_uniform(rng, 60, 700), nodes_hi=rng.randint(10, 64))
        c["ctx_lo"] = max(30, c["ctx_hi"] // 3)
        c["nodes_lo"] = max(8, c["nodes_hi"] // 2)
        c["keep_hi"] = rng.randint(1, c["nodes_lo"] // 2)
        c["hkv"] = min(hkv, 8)
        del c["dtype"], c["hq"]
    return c


# ---------------------------------------------------------------------------------------------- shapes
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _spread(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, _log_uniform(rng, lo, hi)))


def _shapes(case):
    """The lengths of a case: the same for every seed."""
    rng = random.Random(case["shape_seed"])
    op = case["op"]
    s = {}
    if op in ("tree", "sparse", "summarize", "compact"):
        s["base"] = [_spread(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
        if op in ("tree", "compact"):
            s["n"] = [_spread(rng, case["nodes_lo"], case["nodes_hi"]) for _ in s["base"]]
        else:
            s["n"] = [min(b, _spread(rng, case["toks_lo"], case["toks_hi"])) for b in s["base"]]
        # tree, compact: `base` is the prefix; sparse, summarize: `base` is the whole context.
        s["ctx"] = [b + n for b, n in zip(s["base"], s["n"])] if op in ("tree", "compact") else list(s["base"])
        if op == "compact":
            s["keep"] = [rng.randint(1, min(case["keep_hi"], n // 2)) for n in s["n"]]
    else:
        rows = case["groups"] * case["beams"]
        s["prompt"] = [_spread(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["groups"])]
        s["lens"] = []
        for g in range(case["groups"]):
            own_tokens = rng.randint(1, 40)     # generated since the beams parted: the same count for each
            s["lens"] += [s["prompt"][g] + own_tokens] * case["beams"]
        s["parents"] = []
        for g in range(case["groups"]):
            for _ in range(case["beams"]):
                s["parents"].append(g * case["beams"] + rng.randrange(case["beams"]))
        s["rows"] = rows
    return s


# ---------------------------------------------------------------------------------------------- inputs
def _pool_values(gen, shape, dtype, scale):
    """Keys (or values) whose blocks have something in common, as neighbouring tokens do."""
    nb, hkv, bs, d = shape
    x = torch.empty(shape, dtype=torch.bfloat16 if dtype == "bf16" else torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (hkv * bs * d))
    for i in range(0, nb, step):
        m = min(step, nb - i)
        v = torch.randn((m, hkv, bs, d), generator=gen, device=DEV)
        v += torch.randn((m, hkv, 1, d), generator=gen, device=DEV) * 0.7
        if dtype == "bf16":
            x[i:i + m] = v.to(torch.bfloat16)
        else:
            x[i:i + m] = (v / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _tables(gen, counts, num_blocks):
    perm = torch.randperm(num_blocks, generator=gen, device=DEV).to(torch.int32).cpu()
    width = max(counts)
    bt = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(counts):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt.to(DEV)


def _pow2(e):
    """2^e in fp32, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = _shapes(case)
    op, hkv, d = case["op"], case["hkv"], case["d"]
    dtype = case.get("dtype", "bf16")
    st = dict(case=case, shapes=s, k_scale=2.0 ** -6, v_scale=0.0156 if dtype != "bf16" else 1.0)
    if dtype == "bf16":
        st["k_scale"] = 1.0
    if op == "fork":
        _prepare_fork(case, s, st, gen)
    else:
        counts = [_blocks(c) for c in s["ctx"]]
        nb = max(1, int(sum(counts) * 1.1) + 3)
        st["k"] = _pool_values(gen, (nb, hkv, BLOCK, d), dtype, st["k_scale"])
        st["v"] = _pool_values(gen, (nb, hkv, BLOCK, d), dtype, st["v_scale"])
        st["bt"] = _tables(gen, counts, nb)
        st["ctx"] = _i32(s["ctx"])
        st["cu"] = _i32(_cu(s["n"]))
        st["nb"] = nb
        tokens = sum(s["n"])
        if op in ("tree", "sparse"):
            st["scale"] = 1.0 / math.sqrt(d)
            st["q"] = torch.randn((tokens, case["hq"], d), generator=gen, device=DEV).to(torch.bfloat16)
        if op == "tree":
            st["prefix"] = _i32(s["base"])
            st["mask"] = _tree_masks(s["n"], seed, (case["nodes_hi"] + 31) // 32)
        if op in ("sparse", "summarize"):
            st["pos"] = _i32([p for c, n in zip(s["ctx"], s["n"]) for p in range(c - n, c)])
        if op == "sparse":
            codes = torch.zeros((nb, hkv, 2, d), dtype=torch.int8, device=DEV)
            exps = torch.zeros((nb, hkv), dtype=torch.int8, device=DEV)
            st["codes"], st["exps"] = codes, exps
            _plain_bounds(st, (st["bt"] >= 0).nonzero(as_tuple=True))
        if op == "compact":
            _prepare_compact(s, st, seed)
    if own:
        from paged_kv_attention_25_gb300 import pkv
        st["pkv"] = pkv
        st["pool"] = pkv.Pool(st["k"].shape[0], hkv, d, k_storage=st["k"], v_storage=st["v"], dtype=dtype,
                              k_scale=st["k_scale"], v_scale=st["v_scale"])
        if op in ("sparse", "summarize"):
            st["summary"] = pkv.BlockSummary(st["pool"])
            if op == "sparse":
                st["summary"].codes.copy_(st["codes"])
                st["summary"].exps.copy_(st["exps"])
    elif op == "summarize":
        st["codes"] = torch.zeros((st["nb"], hkv, 2, d), dtype=torch.int8, device=DEV)
        st["exps"] = torch.zeros((st["nb"], hkv), dtype=torch.int8, device=DEV)
    return st


def _tree_masks(counts, seed, words):
    """A drafted tree for each request, as rows of bits: bit j of token i's row is set if j is i or an ancestor."""
    rng = random.Random(seed * 7919 + 13)
    rows = []
    for n in counts:
        anc = []
        for i in range(n):
            parent = -1 if i == 0 else rng.randrange(max(-1, i - 9), i)
            anc.append((anc[parent] if parent >= 0 else 0) | (1 << i))
        for a in anc:
            rows.append([((a >> (32 * w)) & 0xFFFFFFFF) for w in range(words)])
    signed = [[x - (1 << 32) if x >= (1 << 31) else x for x in r] for r in rows]
    return torch.tensor(signed, dtype=torch.int32, device=DEV)


def _prepare_fork(case, s, st, gen):
    """Groups of beams that share their prompt's full pages; the last pages are their own."""
    pages = []
    nxt = 0
    for g in range(case["groups"]):
        shared = s["prompt"][g] // BLOCK
        common = list(range(nxt, nxt + shared))
        nxt += shared
        for b in range(case["beams"]):
            n = _blocks(s["lens"][g * case["beams"] + b])
            pages.append(common + list(range(nxt, nxt + n - shared)))
            nxt += n - shared
    spare = s["rows"] * (2 + _blocks(case["room"]))
    nb = nxt + spare + 5
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32).cpu().tolist()
    caps = [n + case["room"] for n in s["lens"]]
    width = max(_blocks(c) for c in caps) + 1
    bt = torch.full((s["rows"], width), -1, dtype=torch.int32)
    refs = torch.zeros(nb, dtype=torch.int32)
    for i, p in enumerate(pages):
        bt[i, :len(p)] = torch.tensor([perm[x] for x in p], dtype=torch.int32)
        for x in p:
            refs[perm[x]] += 1
    shape = (nb, case["hkv"], BLOCK, case["d"])
    st["k"], st["v"] = _pool_values(gen, shape, "bf16", 1.0), _pool_values(gen, shape, "bf16", 1.0)
    st["bt"], st["refs"] = bt.to(DEV), refs.to(DEV)
    st["lens"], st["caps"] = _i32(s["lens"]), _i32(s["lens"])      # the old rows hold pages for their tokens only
    st["parents"] = _i32(s["parents"])
    st["new_caps"] = _i32([s["lens"][p] + case["room"] for p in s["parents"]])
    st["new_bt"] = torch.empty_like(st["bt"])
    st["new_refs"] = torch.empty_like(st["refs"])
    st["nb"] = nb


def _prepare_compact(s, st, seed):
    """The kept drafts of each request: the root, and later slots behind those that they move to."""
    rng = random.Random(seed * 104729 + 5)
    src = []
    for base, n, keep in zip(s["base"], s["n"], s["keep"]):
        src += [base + x for x in [0] + sorted(rng.sample(range(keep, n), keep - 1))]
    st["src"] = _i32(src)
    st["cu_keep"] = _i32(_cu(s["keep"]))
    st["dst"] = _i32(s["base"])


# ---------------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "sparse": _own_sparse, "summarize": _own_summarize, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"tree": _plain_tree, "sparse": _plain_sparse, "summarize": _plain_summarize, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


def _own_tree(st):
    return st["pkv"].pkv_tree_attn(st["pool"], st["q"], st["bt"], st["ctx"], st["prefix"], st["cu"], st["mask"],
                                   st["scale"])


def _own_sparse(st):
    c, p = st["case"], st["pkv"]
    sel = p.pkv_select_blocks(st["pool"], st["summary"], st["q"], st["pos"], st["bt"], st["cu"], c["top_k"],
                              sinks=c["sinks"], recent=c["recent"])
    o, lse = p.pkv_sparse_attn(st["pool"], st["q"], st["pos"], st["bt"], st["cu"], sel, st["scale"])
    return sel, o, lse


def _own_summarize(st):
    s = st["summary"]
    st["pkv"].pkv_summarize(st["pool"], s, st["bt"], st["cu"], st["pos"], st["ctx"])
    return s.codes.float() * _pow2(s.exps)[:, :, None, None]


def _own_fork(st):
    st["pkv"].pkv_fork(st["pool"], st["bt"], st["lens"], st["caps"], st["parents"], st["new_caps"], st["refs"],
                       out_tables=st["new_bt"], out_refs=st["new_refs"])
    return st["new_bt"], st["new_refs"], st["k"], st["v"]


def _own_compact(st):
    st["pkv"].pkv_compact(st["pool"], st["bt"], st["cu_keep"], st["src"], st["dst"])
    return st["k"], st["v"]


# ---------------------------------------------------------------------------------------------- plain forms
def _values(st, which, ids):
    """The blocks `ids` of the pool in fp32: [..., kv heads, 16, head_dim]."""
    x = st[which][ids]
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).float() * st[which + "_scale"]
    return x.float()


def _softmax_rows(s, v):
    """s [..., rows, keys] with -inf where masked, v [..., keys, d] -> (o, lse); empty rows 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z == 0, torch.ones_like(z), z)
    return o, (m + torch.log(z)).squeeze(-1)


def _plain_tree(st):
    # All requests at once, padded to the longest context and the largest tree.
    hkv, d, g = st["case"]["hkv"], st["case"]["d"], st["case"]["hq"] // st["case"]["hkv"]
    bt, ctx, prefix, cu, mask = st["bt"], st["ctx"].long(), st["prefix"].long(), st["cu"].long(), st["mask"]
    reqs, nblk = bt.shape
    n = cu[1:] - cu[:-1]
    nmax = max(st["shapes"]["n"])
    at = torch.arange(nmax, device=DEV)
    valid = at < n[:, None]
    tok = torch.where(valid, cu[:-1, None] + at, 0)
    q = st["q"].float()[tok].view(reqs, nmax, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(reqs, hkv, nmax * g, d)
    ids = bt.clamp(min=0).long()
    k = _values(st, "k", ids).permute(0, 2, 1, 3, 4).reshape(reqs, hkv, nblk * BLOCK, d)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    j = torch.arange(nblk * BLOCK, device=DEV)
    bit = (j - prefix[:, None])[:, None, :].expand(reqs, nmax, -1)
    word = torch.gather(mask.long()[tok], 2, bit.clamp(0, mask.shape[1] * 32 - 1) // 32)
    seen = (bit < 0) | (((word >> (bit.clamp(min=0) % 32)) & 1) != 0)
    seen = seen & (j < ctx[:, None])[:, None, :] & valid[:, :, None]
    s = s.view(reqs, hkv, nmax, g, -1).masked_fill(~seen[:, None, :, None, :], -math.inf).view(reqs, hkv, nmax * g, -1)
    v = _values(st, "v", ids).permute(0, 2, 1, 3, 4).reshape(reqs, hkv, nblk * BLOCK, d)
    o, lse = _softmax_rows(s, v)
    o = o.view(reqs, hkv, nmax, g, d).permute(0, 2, 1, 3, 4).reshape(reqs, nmax, hkv * g, d)
    lse = lse.view(reqs, hkv, nmax, g).permute(0, 2, 1, 3).reshape(reqs, nmax, hkv * g)
    req = torch.repeat_interleave(torch.arange(reqs, device=DEV), n, output_size=st["q"].shape[0])
    row = torch.arange(st["q"].shape[0], device=DEV) - cu[req]
    return o[req, row].to(torch.bfloat16), lse[req, row]


def _plain_bounds(st, at):
    """The bounds of block at[1][i] of request at[0][i], for all i, into codes [blocks][kv heads][upper, lower][d] and
    exps [blocks][kv heads]."""
    req, blk = at
    ids = st["bt"][req, blk].long()
    x = st["k"][ids]
    x = x.view(torch.float8_e4m3fn).float() if x.dtype == torch.uint8 else x.float()
    past = blk[:, None] * BLOCK + torch.arange(BLOCK, device=DEV) >= st["ctx"].long()[req][:, None]
    hi = x.masked_fill(past[:, None, :, None], -math.inf).amax(2)
    lo = x.masked_fill(past[:, None, :, None], math.inf).amin(2)
    mant, e = torch.frexp(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    e = torch.where(mant <= 127.0 / 128.0, e - 7, e - 6).clamp(min=-126)
    inv = _pow2(-e)[:, :, None]
    st["codes"][ids] = torch.stack([torch.ceil(hi * inv), torch.floor(lo * inv)], 2).to(torch.int8)
    st["exps"][ids] = e.to(torch.int8)


def _plain_summarize(st):
    cu, pos = st["cu"].long(), st["pos"].long()
    req = torch.repeat_interleave(torch.arange(cu.shape[0] - 1, device=DEV), cu[1:] - cu[:-1], output_size=pos.shape[0])
    opens = ((pos % BLOCK == 0) | (torch.arange(pos.shape[0], device=DEV) == cu[req])).nonzero()[:, 0]
    _plain_bounds(st, (req[opens], pos[opens] // BLOCK))
    return st["codes"].float() * _pow2(st["exps"])[:, :, None, None]


def _plain_sparse(st):
    c = st["case"]
    hkv, d, g, topk = c["hkv"], c["d"], c["hq"] // c["hkv"], c["top_k"]
    bt, cu, pos = st["bt"].long(), st["cu"].long(), st["pos"].long()
    tokens, nblk = pos.shape[0], bt.shape[1]
    req = torch.repeat_interleave(torch.arange(bt.shape[0], device=DEV), cu[1:] - cu[:-1], output_size=tokens)
    q = st["q"].float().view(tokens, hkv, g, d)
    # Whole-number queries, summed over the heads of a group by sign.
    most = 32767 // g
    mant, e = torch.frexp(q.abs().amax((2, 3)))
    ml, el = math.frexp(most)
    f = torch.where(mant <= ml, e - el, e - el + 1)
    qi = torch.round(q * _pow2(-f)[:, :, None, None])
    both = torch.cat([qi.clamp(min=0).sum(2), qi.clamp(max=0).sum(2)], -1).double()        # [T, hkv, 2d]
    # In 64 bits the sums are whole numbers without rounding: the order of the blocks is exact.
    score = torch.empty((tokens, hkv, nblk), device=DEV)
    for r in range(bt.shape[0]):
        a, b = _token_range(st, r)
        ids = bt[r].clamp(min=0)
        w = st["codes"][ids].reshape(nblk, hkv, 2 * d).permute(1, 2, 0).double()
        dots = torch.matmul(both[a:b].transpose(0, 1), w)                                     # [hkv, n, nblk]
        score[a:b] = (dots.float() * _pow2(st["exps"][ids].t())[:, None, :]).transpose(0, 1)
    last = pos // BLOCK
    j = torch.arange(nblk, device=DEV)
    seen = j <= last[:, None]
    always = seen & ((j < c["sinks"]) | (j > (last - c["recent"])[:, None]))
    score = score.masked_fill(always[:, None], math.inf).masked_fill(~seen[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :topk]
    order = torch.where(order <= last[:, None, None], order, nblk).sort(-1)[0]
    sel = torch.where(order < nblk, order, -1)
    if sel.shape[-1] < topk:
        sel = torch.cat([sel, sel.new_full((tokens, hkv, topk - sel.shape[-1]), -1)], -1)
    # Attention over the listed blocks.
    ids = torch.gather(bt[req][:, None].expand(-1, hkv, -1), 2, sel.clamp(min=0)).clamp(min=0)
    head = torch.arange(hkv, device=DEV)[:, None]
    k = _values(st, "k", (ids, head)).reshape(tokens, hkv, topk * BLOCK, d)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    key = (sel[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)).reshape(tokens, hkv, -1)
    ok = (key >= 0) & (key <= pos[:, None, None]) & (sel >= 0).repeat_interleave(BLOCK, -1)
    s = s.masked_fill(~ok[:, :, None, :], -math.inf)
    v = _values(st, "v", (ids, head)).reshape(tokens, hkv, topk * BLOCK, d)
    o, lse = _softmax_rows(s, v)
    return sel.to(torch.int32), o.reshape(tokens, hkv * g, d).to(torch.bfloat16), lse.reshape(tokens, hkv * g)


def _token_range(st, r):
    a = sum(st["shapes"]["n"][:r])
    return a, a + st["shapes"]["n"][r]


def _plain_fork(st):
    bt, lens, caps = st["bt"].long(), st["lens"].long(), st["caps"].long()
    parents, new_caps = st["parents"].long(), st["new_caps"].long()
    rows, width = bt.shape
    nb = st["refs"].shape[0]
    j = torch.arange(width, device=DEV)
    kids = torch.bincount(parents.clamp(min=0), weights=(parents >= 0).float(), minlength=rows).long()
    full, part = lens // BLOCK, lens % BLOCK
    # 1. Full pages: one holder less for the old row, one more for each child; the last, partly filled page of a
    #    continued row is settled afterwards.
    delta = torch.where(j < full[:, None], (kids - 1)[:, None], -1)
    settle = (part > 0) & (kids > 0)
    held = (j < ((caps + BLOCK - 1) // BLOCK)[:, None]) & ~(settle[:, None] & (j == full[:, None]))
    refs = st["refs"].long().clone()
    refs.index_add_(0, torch.where(held, bt, 0).view(-1), torch.where(held, delta, 0).view(-1))
    # 2. Its lowest child keeps that page if nobody else holds it; every other child copies it.
    last = torch.gather(bt, 1, full.clamp(max=width - 1)[:, None])[:, 0].clamp(min=0)
    alone = settle & (refs[last] == 1)
    child = torch.arange(parents.shape[0], device=DEV)
    first = torch.full((rows,), parents.shape[0], device=DEV).scatter_reduce_(
        0, parents.clamp(min=0), torch.where(parents >= 0, child, parents.shape[0]), "amin")
    p = parents.clamp(min=0)
    has = parents >= 0
    keeps = has & alone[p] & (first[p] == child)
    copies = has & (part[p] > 0) & ~keeps
    # 3. Fresh pages: the lowest ones without a holder, in the order of children and of their pages.
    shared = torch.where(has, full[p] + keeps.long(), 0)
    total = (torch.maximum(new_caps, torch.where(has, lens[p], 0)) + BLOCK - 1) // BLOCK
    need = (total - shared).clamp(min=0)
    start = torch.cumsum(need, 0) - need
    free = torch.sort(torch.where(refs == 0, torch.arange(nb, device=DEV), nb))[0]
    fresh = (j >= shared[:, None]) & (j < total[:, None])
    which = (start[:, None] + j - shared[:, None]).clamp(0, nb - 1)
    new = torch.where(j < shared[:, None], bt[p], torch.where(fresh, free[which], -1))
    refs.index_add_(0, torch.where(fresh, new, 0).view(-1), fresh.long().view(-1))
    refs.index_add_(0, last, -(settle & ~alone).long())
    # 4. The copies: the rows that hold tokens.
    src = last[p]
    dst = torch.gather(new, 1, full[p].clamp(max=width - 1)[:, None])[:, 0]
    at = copies.nonzero()[:, 0]
    src, dst = src[at], dst[at]
    take = (torch.arange(BLOCK, device=DEV) < part[p][at][:, None])[:, None, :, None]
    for x in (st["k"], st["v"]):
        x[dst] = torch.where(take, x[src], x[dst])
    st["new_bt"].copy_(new)
    st["new_refs"].copy_(refs)
    return st["new_bt"], st["new_refs"], st["k"], st["v"]


def _plain_compact(st):
    bt, cu, src = st["bt"].long(), st["cu_keep"].long(), st["src"].long()
    n = src.shape[0]
    req = torch.repeat_interleave(torch.arange(bt.shape[0], device=DEV), cu[1:] - cu[:-1], output_size=n)
    dst = st["dst"].long()[req] + torch.arange(n, device=DEV) - cu[req]
    sp, dp = bt[req, src // BLOCK], bt[req, dst // BLOCK]
    for x in (st["k"], st["v"]):
        x[dp, :, dst % BLOCK] = x[sp, :, src % BLOCK]
    return st["k"], st["v"]


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"tree": _exact_tree, "sparse": _exact_sparse, "summarize": _exact_summarize, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](case, st)


def _pow2_wide(e):
    """2^e in 64 bits, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _wide(st, which, ids):
    x = st[which][ids.long()]
    x = x.view(torch.float8_e4m3fn).double() if x.dtype == torch.uint8 else x.double()
    return x * st[which + "_scale"]


def _one_head(q, k, v, seen, scale):
    """q [rows, d], k and v [keys, d], seen [rows, keys], all in 64 bits."""
    s = (q @ k.t()) * scale
    s[~seen] = -math.inf
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return w @ v, lse


def _exact_tree(case, st):
    hkv, g, d = case["hkv"], case["hq"] // case["hkv"], case["d"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    bits = st["mask"].cpu().tolist()
    for r, (base, n, ctx) in enumerate(zip(st["shapes"]["base"], st["shapes"]["n"], st["shapes"]["ctx"])):
        a, b = _token_range(st, r)
        ids = st["bt"][r, :_blocks(ctx)]
        k = _wide(st, "k", ids).permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :ctx]
        v = _wide(st, "v", ids).permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :ctx]
        tree = [[bool((bits[a + i][x // 32] >> (x % 32)) & 1) for x in range(n)] for i in range(n)]
        seen = torch.ones((n, ctx), dtype=torch.bool, device=DEV)
        seen[:, base:] = torch.tensor(tree, device=DEV)
        seen = seen.repeat_interleave(g, 0)
        for h in range(hkv):
            rows = st["q"][a:b, h * g:(h + 1) * g].double().reshape(n * g, d)
            oo, ll = _one_head(rows, k[h], v[h], seen, st["scale"])
            o[a:b, h * g:(h + 1) * g] = oo.view(n, g, d)
            lse[a:b, h * g:(h + 1) * g] = ll.view(n, g)
    return o, lse


def _power_for(amax, most):
    """The smallest power of two p with amax <= most * p, by trial."""
    if amax == 0.0:
        return 1.0
    p = 2.0 ** math.floor(math.log2(amax / most))
    while amax > most * p:
        p *= 2.0
    while amax <= most * (p / 2.0):
        p /= 2.0
    return p


def _exact_sparse(case, st):
    hkv, g, d, topk = case["hkv"], case["hq"] // case["hkv"], case["d"], case["top_k"]
    tokens = st["q"].shape[0]
    sel = torch.full((tokens, hkv, topk), -1, dtype=torch.int32)
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    pos = st["pos"].tolist()
    most = 32767 // g
    amax = st["q"].double().view(tokens, hkv, g * d).abs().amax(-1).tolist()
    for r in range(len(st["shapes"]["ctx"])):
        a, b = _token_range(st, r)
        for t in range(a, b):
            blocks = pos[t] // BLOCK + 1
            ids = st["bt"][r, :blocks].long()
            up = st["codes"][ids].double()
            power = _pow2_wide(st["exps"][ids])
            forced = [x for x in range(blocks) if x < case["sinks"] or x >= blocks - case["recent"]]
            for h in range(hkv):
                qh = st["q"][t, h * g:(h + 1) * g].double()
                qi = torch.round(qh / _power_for(amax[t][h], most))
                whole = (up[:, h, 0] @ qi.clamp(min=0).sum(0)) + (up[:, h, 1] @ qi.clamp(max=0).sum(0))
                key = whole.float().double() * power[:, h]
                key[forced] = math.inf
                rank = torch.argsort(-key, stable=True)[:topk].sort()[0]
                sel[t, h, :rank.shape[0]] = rank.to(torch.int32).cpu()
                kk = _wide_head(st, "k", ids[rank], h)
                vv = _wide_head(st, "v", ids[rank], h)
                at = (rank[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).reshape(-1)
                seen = (at <= pos[t])[None].expand(g, -1)
                o[t, h * g:(h + 1) * g], lse[t, h * g:(h + 1) * g] = _one_head(qh, kk, vv, seen, st["scale"])
    return sel.to(DEV), o, lse


def _wide_head(st, which, ids, h):
    x = st[which][ids, h]
    x = x.view(torch.float8_e4m3fn).double() if x.dtype == torch.uint8 else x.double()
    return (x * st[which + "_scale"]).reshape(-1, x.shape[-1])


def _exact_summarize(case, st):
    out = torch.zeros((st["nb"], case["hkv"], 2, case["d"]), dtype=torch.float64, device=DEV)
    for r, (ctx, n) in enumerate(zip(st["shapes"]["ctx"], st["shapes"]["n"])):
        for j in range((ctx - n) // BLOCK, _blocks(ctx)):
            block = int(st["bt"][r, j])
            x = st["k"][block, :, :min(BLOCK, ctx - j * BLOCK)]
            x = x.view(torch.float8_e4m3fn).double() if x.dtype == torch.uint8 else x.double()
            amax = x.abs().amax((1, 2))
            e = torch.ceil(torch.log2(torch.clamp(amax, min=2.0 ** -126) / 127.0))
            e = torch.where(amax > 127.0 * _pow2_wide(e), e + 1.0, e)       # the logarithm may be off at a border
            e = torch.where(amax <= 127.0 * _pow2_wide(e - 1.0), e - 1.0, e)
            unit = _pow2_wide(e.clamp(min=-126.0))[:, None]
            out[block, :, 0] = torch.ceil(x.amax(1) / unit) * unit
            out[block, :, 1] = torch.floor(x.amin(1) / unit) * unit
    return out


def _exact_fork(case, st):
    tables, refs = st["bt"].tolist(), st["refs"].tolist()
    lens, caps = st["lens"].tolist(), st["caps"].tolist()
    parents, new_caps = st["parents"].tolist(), st["new_caps"].tolist()
    width = len(tables[0])
    new = [[-1] * width for _ in parents]
    kids = [[i for i, p in enumerate(parents) if p == r] for r in range(len(lens))]
    for r, row in enumerate(tables):                      # every page loses its old holders but a continued part page
        for j in range(_blocks(caps[r])):
            if not (kids[r] and lens[r] % BLOCK and j == lens[r] // BLOCK):
                refs[row[j]] -= 1
        for i in kids[r]:
            for j in range(lens[r] // BLOCK):
                new[i][j] = row[j]
                refs[row[j]] += 1
    drop, copy = [], []
    state = list(refs)
    for r, row in enumerate(tables):
        at = lens[r] // BLOCK
        if kids[r] and lens[r] % BLOCK:
            if state[row[at]] == 1:
                new[kids[r][0]][at] = row[at]
                copy += [(i, r) for i in kids[r][1:]]
            else:
                drop.append(row[at])
                copy += [(i, r) for i in kids[r]]
    free = iter([b for b in range(len(refs)) if refs[b] == 0])
    for i, p in enumerate(parents):
        want = _blocks(max(new_caps[i], lens[p] if p >= 0 else 0))
        for j in range(want):
            if new[i][j] < 0:
                new[i][j] = next(free)
                refs[new[i][j]] = 1
    for b in drop:
        refs[b] -= 1
    k, v = st["k"], st["v"]
    for i, r in copy:
        at, rows = lens[r] // BLOCK, lens[r] % BLOCK
        for x in (k, v):
            x[new[i][at], :, :rows] = x[tables[r][at], :, :rows]
    return (torch.tensor(new, dtype=torch.int32, device=DEV), torch.tensor(refs, dtype=torch.int32, device=DEV),
            k.double(), v.double())


def _exact_compact(case, st):
    src, cu, dst = st["src"].tolist(), st["cu_keep"].tolist(), st["dst"].tolist()
    bt = st["bt"].tolist()
    for x in (st["k"], st["v"]):
        for r in range(len(dst)):
            for i in range(cu[r], cu[r + 1]):
                a, b = src[i], dst[r] + i - cu[r]
                if a != b:
                    x[bt[r][b // BLOCK], :, b % BLOCK] = x[bt[r][a // BLOCK], :, a % BLOCK]
    return st["k"].double(), st["v"].double()


# ---------------------------------------------------------------------------------------------- work
def work(case):
    s = _shapes(case)
    hkv, d = case["hkv"], case["d"]
    e = 1 if case.get("dtype") == "fp8_e4m3" else 2
    row = hkv * d * e                               # one token's K (or V)
    if case["op"] == "tree":
        tokens = sum(s["n"])
        return {"bytes": 2 * row * sum(s["ctx"]) + tokens * case["hq"] * (4 * d + 4) + tokens * 4,
                "flops": sum(4 * d * case["hq"] * (n * base + n) for n, base in zip(s["n"], s["base"]))}
    if case["op"] == "sparse":
        tokens, keys = sum(s["n"]), [min(case["top_k"] * BLOCK, c) for c in s["ctx"]]
        bounds = sum(_blocks(c) for c in s["ctx"])
        return {"bytes": bounds * hkv * (2 * d + 1) + 2 * row * sum(keys) + tokens * case["hq"] * (4 * d + 4)
                + tokens * hkv * case["top_k"] * 4,
                "flops": sum(n * (4 * d * case["hq"] * k + 4 * d * hkv * _blocks(c))
                             for n, k, c in zip(s["n"], keys, s["ctx"]))}
    if case["op"] == "summarize":
        firsts = [(c - n) // BLOCK for c, n in zip(s["ctx"], s["n"])]
        keys = sum(c - f * BLOCK for c, f in zip(s["ctx"], firsts))
        blocks = sum(_blocks(c) - f for c, f in zip(s["ctx"], firsts))
        return {"bytes": row * keys + blocks * hkv * (2 * d + 1), "flops": 2 * d * hkv * keys}
    if case["op"] == "fork":
        # Every old entry is read, every new one written; the copied part pages are what is not kept.
        old, new = sum(_blocks(n) for n in s["lens"]), sum(_blocks(s["lens"][p] + case["room"]) for p in s["parents"])
        copies = len(s["parents"]) - len(set(s["parents"]))
        part = sum(n % BLOCK for n in s["lens"]) / len(s["lens"])
        return {"bytes": int(4 * (old + new) + copies * part * row * 4), "flops": old + new}
    kept = sum(s["keep"])
    return {"bytes": kept * (row * 4 + 4), "flops": kept}
