"""What is measured of the 8-bit cache and of attention with modified scores.

The pool is [blocks][kv heads][16][head_dim] in bf16, in e4m3 codes with one scale for K and one for V, or in int8 codes
with a power of two for each (block, kv head) of K and of V: a code c stands for c * 2^e, |c| <= 127.

  write   new rows are quantised into the blocks of their requests; a block's exponent is the larger of the one it has (if
          it holds tokens) and the smallest that fits the new rows, and held codes follow it.  The rows of the written
          blocks are then read back.
  read    rows of a cache as contiguous bf16.
  attn    attention of one or more tokens a request over the cache, scores capped by a tanh or lowered by a slope times
          the distance, keys limited to a window, a document or a prefix.

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
        # A decode step of one conversation: one row joins the last block.
        dict(name="write_one_user", op="write", reqs=1, ctx_lo=190, ctx_hi=240, toks_lo=1, toks_hi=1, hq=8, hkv=2, d=64,
             dtype="int8", shape_seed=1),
        # A decode step of a batch, some requests with a few accepted drafts: blocks that hold tokens already.
        dict(name="write_batch", op="write", reqs=128, ctx_lo=100, ctx_hi=4000, toks_lo=1, toks_hi=5, hq=64, hkv=8, d=128,
             dtype="int8", shape_seed=2),
        # Prompts of a batch are stored: bound by memory.
        dict(name="write_prompts", op="write", reqs=6, ctx_lo=3000, ctx_hi=9000, toks_lo=9000, toks_hi=9000, hq=64, hkv=8,
             d=128, dtype="int8", shape_seed=3),
        # The last tokens of a few conversations are looked at.
        dict(name="read_tails", op="read", reqs=3, ctx_lo=60, ctx_hi=300, toks_lo=1, toks_hi=40, hq=8, hkv=2, d=64,
             dtype="int8", shape_seed=4),
        # Whole conversations leave the 8-bit cache for one of another type.
        dict(name="read_conversations", op="read", reqs=12, ctx_lo=500, ctx_hi=9000, toks_lo=9000, toks_hi=9000, hq=64,
             hkv=8, d=128, dtype="int8", shape_seed=5),
        # One conversation of a small model, one token, over the 8-bit cache: latency.
        dict(name="int8_one_user", op="attn", reqs=1, ctx_lo=2900, ctx_hi=3050, toks_lo=1, toks_hi=1, hq=8, hkv=2, d=64,
             dtype="int8", shape_seed=6),
        # Decode of a batch of ragged contexts with grouped heads over the 8-bit cache: bound by reading it.
        dict(name="int8_decode", op="attn", reqs=64, ctx_lo=500, ctx_hi=33000, toks_lo=1, toks_hi=1, hq=64, hkv=8, d=128,
             dtype="int8", shape_seed=7),
        # New turns behind cached history, of very different lengths, over the 8-bit cache.
        dict(name="int8_new_turns", op="attn", reqs=10, ctx_lo=1000, ctx_hi=12000, toks_lo=1, toks_hi=1500, hq=64, hkv=8,
             d=128, dtype="int8", shape_seed=8),
        # Prompts of a model that caps its scores.
        dict(name="cap_prompts", op="attn", reqs=4, ctx_lo=1500, ctx_hi=6000, toks_lo=6000, toks_hi=6000, hq=64, hkv=8,
             d=128, dtype="bf16", softcap=30.0, shape_seed=9),
        # Decode with a bias that falls with the distance, a key head for each query head, e4m3 cache.
        dict(name="distance_decode", op="attn", reqs=32, ctx_lo=300, ctx_hi=8000, toks_lo=1, toks_hi=1, hq=40, hkv=40,
             d=128, dtype="fp8_e4m3", slopes=True, shape_seed=10),
        # Layers with a sliding window and four tokens that are always seen, capped scores, a few tokens a request: the
        # contexts are far longer than what is read.
        dict(name="window_steps", op="attn", reqs=48, ctx_lo=9000, ctx_hi=60000, toks_lo=1, toks_hi=4, hq=64, hkv=8, d=128,
             dtype="bf16", softcap=50.0, window=4096, prefix="sinks", shape_seed=11),
        # Packed documents behind a common prefix that is seen both ways, small model.
        dict(name="packed_documents", op="attn", reqs=3, ctx_lo=700, ctx_hi=2800, toks_lo=6000, toks_hi=6000, hq=8, hkv=2,
             d=64, dtype="bf16", docs=True, prefix="third", shape_seed=12),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "attn"])
    hkv, group = rng.choice([(1, 8), (2, 1), (2, 4), (3, 5), (4, 2), (8, 1), (8, 8), (5, 1), (40, 1), (8, 4), (1, 24)])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=rng.choice([64, 128, 128]), dtype="int8", shape_seed=rng.randrange(1 << 30))
    if op != "attn":
        if op == "read":
            c["dtype"] = rng.choice(["int8", "int8", "bf16", "fp8_e4m3"])
        hi = _log_uniform(rng, 1, 9000)
        c["reqs"] = max(1, min(_log_uniform(rng, 1, 128), 200_000 // (hkv * hi)))
        c["ctx_hi"], c["ctx_lo"] = hi, max(1, hi // rng.choice([1, 4, 20]))
        c["toks_hi"] = _log_uniform(rng, 1, hi)
        c["toks_lo"] = max(1, c["toks_hi"] // rng.choice([1, 3, 10]))
        return c
    c["dtype"] = rng.choice(["int8", "int8", "int8", "bf16", "bf16", "fp8_e4m3"])
    prompt = rng.random() < 0.5
    if prompt:
        hi = _log_uniform(rng, 16, 6000)
        most = 64 * 2.0e7 / (c["hq"] * hi)           # new tokens of the batch, so that the pairs stay below the listed ones'
        c["toks_hi"] = int(max(1, min(_log_uniform(rng, 4, hi), most)))
        c["reqs"] = int(max(1, min(_log_uniform(rng, 1, 16), most // c["toks_hi"])))
    else:
        hi = _log_uniform(rng, 1, 60000)
        c["toks_hi"] = min(rng.choice([1, 1, 2, 7]), hi)
        c["reqs"] = max(1, min(_log_uniform(rng, 1, 64), 1_500_000 // (hkv * hi)))
    c["ctx_hi"], c["ctx_lo"] = hi, max(1, hi // rng.choice([1, 2, 10, 50]))
    c["toks_lo"] = max(1, c["toks_hi"] // rng.choice([1, 2, 20]))
    if rng.random() < 0.6:
        if rng.random() < 0.4:
            c["softcap"] = rng.choice([5.0, 30.0, 50.0])
        if rng.random() < 0.4:
            c["slopes"] = True
        if rng.random() < 0.4:
            c["window"] = _log_uniform(rng, 1, max(2, hi))
        if rng.random() < 0.3:
            c["docs"] = True
        if rng.random() < 0.4:
            c["prefix"] = rng.choice(["sinks", "third"])
    return c


# ---------------------------------------------------------------------------------------------- shapes
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _spread(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, _log_uniform(rng, lo, hi)))


def _shapes(case):
    """The lengths of a case: the same for every seed.  n of the ctx tokens of a request are new."""
    rng = random.Random(case["shape_seed"])
    s = {"ctx": [_spread(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]}
    s["n"] = [min(c, _spread(rng, case["toks_lo"], case["toks_hi"])) for c in s["ctx"]]
    kind = case.get("prefix")
    s["prefix"] = [min(c, 4) if kind == "sinks" else c // 3 if kind == "third" else 0 for c in s["ctx"]]
    if case.get("docs"):
        s["first"] = []
        for ctx, n, pre in zip(s["ctx"], s["n"], s["prefix"]):
            starts, at = [], pre
            while at < ctx:
                starts.append(at)
                at += _log_uniform(rng, 30, 1500)
            k = 0
            for p in range(ctx - n, ctx):
                while k + 1 < len(starts) and starts[k + 1] <= p:
                    k += 1
                s["first"].append(starts[k] if starts and p >= starts[k] else 0)
    return s


# ---------------------------------------------------------------------------------------------- inputs
def _pow2(e):
    """2^e in fp32, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _least_exponent(amax):
    """The smallest e >= -126 with amax <= 127 * 2^e."""
    mant, e = torch.frexp(amax)
    return torch.where(mant <= 127.0 / 128.0, e - 7, e - 6).clamp(min=-126)


def _normal(gen, shape, spread):
    """Rows as a model makes them: some heads and tokens louder than others."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return x * torch.exp(torch.randn(shape[:-1] + (1,), generator=gen, device=DEV) * spread)


def _pool_values(gen, shape, dtype, scale):
    """A filled pool: values (bf16), codes (uint8), or codes and exponents (int8)."""
    nb, hkv, bs, d = shape
    x = torch.empty(shape, dtype={"bf16": torch.bfloat16, "fp8_e4m3": torch.uint8, "int8": torch.int8}[dtype], device=DEV)
    exps = torch.zeros((nb, hkv), dtype=torch.int8, device=DEV) if dtype == "int8" else None
    step = max(1, (1 << 25) // (hkv * bs * d))
    for i in range(0, nb, step):
        v = _normal(gen, (min(step, nb - i), hkv, bs, d), 0.3).to(torch.bfloat16)
        if dtype == "bf16":
            x[i:i + step] = v
        elif dtype == "int8":
            e = _least_exponent(v.float().abs().amax((2, 3)))
            x[i:i + step] = torch.round(v.float() * _pow2(-e)[:, :, None, None]).to(torch.int8)
            exps[i:i + step] = e.to(torch.int8)
        else:
            x[i:i + step] = (v.float() / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    return x, exps


def _tables(gen, counts, num_blocks):
    perm = torch.randperm(num_blocks, generator=gen, device=DEV).to(torch.int32).cpu()
    bt = torch.full((len(counts), max(counts)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(counts):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt.to(DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _touched(s):
    """First position of the first written block of each request."""
    return [(c - n) // BLOCK * BLOCK for c, n in zip(s["ctx"], s["n"])]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = _shapes(case)
    hkv, d, dtype = case["hkv"], case["d"], case["dtype"]
    fp8 = dtype == "fp8_e4m3"
    st = dict(case=case, shapes=s, k_scale=2.0 ** -6 if fp8 else 1.0, v_scale=0.0156 if fp8 else 1.0)
    counts = [_blocks(c) for c in s["ctx"]]
    nb = max(1, int(sum(counts) * 1.1) + 3)
    st["k"], st["k_exps"] = _pool_values(gen, (nb, hkv, BLOCK, d), dtype, st["k_scale"])
    st["v"], st["v_exps"] = _pool_values(gen, (nb, hkv, BLOCK, d), dtype, st["v_scale"])
    st["bt"] = _tables(gen, counts, nb)
    st["ctx"] = _i32(s["ctx"])
    st["cu"] = _i32(_cu(s["n"]))
    st["pos"] = _i32([p for c, n in zip(s["ctx"], s["n"]) for p in range(c - n, c)])
    tokens = sum(s["n"])
    if case["op"] == "write":
        st["held"] = _i32([c - n for c, n in zip(s["ctx"], s["n"])])
        st["k_new"] = _normal(gen, (tokens, hkv, d), 0.5).to(torch.bfloat16)
        st["v_new"] = _normal(gen, (tokens, hkv, d), 0.5).to(torch.bfloat16)
        st["back_pos"] = _i32([p for c, f in zip(s["ctx"], _touched(s)) for p in range(f, c)])
        st["back_cu"] = _i32(_cu([c - f for c, f in zip(s["ctx"], _touched(s))]))
    if case["op"] == "attn":
        st["scale"] = 1.0 / math.sqrt(d)
        st["q"] = torch.randn((tokens, case["hq"], d), generator=gen, device=DEV).to(torch.bfloat16)
        if case.get("slopes"):
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["hq"]) for h in range(case["hq"])],
                                        dtype=torch.float32, device=DEV)
        if case.get("docs"):
            st["first"] = _i32(s["first"])
        if case.get("prefix"):
            st["prefix"] = _i32(s["prefix"])
    if own:
        from paged_kv_attention_25_gb300 import pkv
        st["pkv"] = pkv
        extra = dict(k_exps=st["k_exps"], v_exps=st["v_exps"]) if dtype == "int8" else {}
        st["pool"] = pkv.Pool(nb, hkv, d, k_storage=st["k"], v_storage=st["v"], dtype=dtype, k_scale=st["k_scale"],
                              v_scale=st["v_scale"], **extra)
    return st


# ---------------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "attn": _own_attn}[op](state)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn}[op](state)


def _own_write(st):
    p = st["pkv"]
    p.pkv_append_int8(st["pool"], st["bt"], st["cu"], st["pos"], st["held"], st["k_new"], st["v_new"])
    k, v = p.pkv_read_rows(st["pool"], st["bt"], st["back_cu"], st["back_pos"])
    return k, v, st["k_exps"], st["v_exps"]


def _own_read(st):
    return st["pkv"].pkv_read_rows(st["pool"], st["bt"], st["cu"], st["pos"])


def _own_attn(st):
    c = st["case"]
    return st["pkv"].pkv_score_attn(st["pool"], st["q"], st["pos"], st["bt"], st["ctx"], st["cu"], st["scale"],
                                    softcap=c.get("softcap", 0.0), window=c.get("window", 0), slopes=st.get("slopes"),
                                    first_keys=st.get("first"), prefix_lens=st.get("prefix"))


# ---------------------------------------------------------------------------------------------- plain forms
def _req_of(cu, tokens):
    n = cu[1:] - cu[:-1]
    return torch.repeat_interleave(torch.arange(n.shape[0], device=DEV), n, output_size=tokens)


def _rows(st, which, ids, slots):
    """Rows `slots` of blocks `ids` in fp32: [n, kv heads, d]."""
    x = st[which][ids, :, slots]
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).float() * st[which + "_scale"]
    if x.dtype == torch.int8:
        return x.float() * _pow2(st[which + "_exps"][ids])[..., None]
    return x.float()


def _read(st, cu, pos):
    pos = pos.long()
    ids = st["bt"].long()[_req_of(cu.long(), pos.shape[0]), pos // BLOCK]
    return tuple(_rows(st, which, ids, pos % BLOCK).to(torch.bfloat16) for which in ("k", "v"))


def _plain_read(st):
    return _read(st, st["cu"], st["pos"])


def _plain_write(st):
    pos, cu, held = st["pos"].long(), st["cu"].long(), st["held"].long()
    req = _req_of(cu, pos.shape[0])
    opens = (pos % BLOCK == 0) | (torch.arange(pos.shape[0], device=DEV) == cu[req])      # the first new row of a block
    block = torch.cumsum(opens.long(), 0) - 1                # of each row, among the written ones
    lead = opens.nonzero()[:, 0]
    ids = st["bt"].long()[req[lead], pos[lead] // BLOCK]
    holds = (pos[lead] // BLOCK * BLOCK < held[req[lead]])[:, None]
    for x, name in ((st["k_new"].float(), "k"), (st["v_new"].float(), "v")):
        codes, exps = st[name], st[name + "_exps"]
        amax = torch.zeros((lead.shape[0], x.shape[1]), device=DEV).index_reduce_(0, block, x.abs().amax(-1), "amax")
        old, e = exps[ids].int(), _least_exponent(amax)
        e = torch.where(holds, torch.maximum(old, e), e)
        less = torch.where(holds, old - e, torch.zeros_like(e)).clamp(min=-126)
        codes[ids] = torch.round(codes[ids].float() * _pow2(less)[..., None, None]).to(torch.int8)
        exps[ids] = e.to(torch.int8)
        codes[ids[block], :, pos % BLOCK] = torch.round(x * _pow2(-e[block])[..., None]).to(torch.int8)
    return _read(st, st["back_cu"], st["back_pos"]) + (st["k_exps"], st["v_exps"])


def _plain_attn(st):
    c, s = st["case"], st["shapes"]
    hkv, d, g = c["hkv"], c["d"], c["hq"] // c["hkv"]
    tokens = st["q"].shape[0]
    o = torch.empty((tokens, c["hq"], d), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((tokens, c["hq"]), device=DEV)
    first = 0
    for r, (ctx, n) in enumerate(zip(s["ctx"], s["n"])):
        j = torch.arange(ctx, device=DEV)
        ids = st["bt"][r].long()[j // BLOCK]
        k = _rows(st, "k", ids, j % BLOCK).permute(1, 2, 0)
        v = _rows(st, "v", ids, j % BLOCK).transpose(0, 1)
        step = max(1, (1 << 28) // (c["hq"] * ctx))
        for a in range(first, first + n, step):
            b = min(first + n, a + step)
            p = st["pos"][a:b].long()[:, None]
            q = st["q"][a:b].float().view(b - a, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, (b - a) * g, d)
            x = (torch.matmul(q, k) * st["scale"]).view(hkv, b - a, g, ctx)
            if c.get("softcap"):
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if "slopes" in st:
                x = x - st["slopes"].view(hkv, 1, g, 1) * (p - j).abs().float()[:, None]
            seen = j <= p
            if c.get("window"):
                seen = seen & (j > p - c["window"])
            if "first" in st:
                seen = seen & (j >= st["first"][a:b].long()[:, None])
            if "prefix" in st:
                seen = seen | (j < st["prefix"][r])
            x = x.masked_fill(~seen[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            w = torch.exp(x - m)
            z = w.sum(-1, keepdim=True)
            y = torch.matmul(w.view(hkv, (b - a) * g, ctx), v).view(hkv, b - a, g, d) / torch.where(z == 0, torch.ones_like(z), z)
            o[a:b] = y.permute(1, 0, 2, 3).reshape(b - a, c["hq"], d).to(torch.bfloat16)
            lse[a:b] = (m + torch.log(z)).squeeze(-1).permute(1, 0, 2).reshape(b - a, c["hq"])
        first += n
    return o, lse


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn}[case["op"]](case, st)


def _wide_pool(st, which):
    """The value of every slot of the pool."""
    x = st[which]
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).double() * st[which + "_scale"]
    if x.dtype == torch.int8:
        return torch.ldexp(x.double(), st[which + "_exps"].int()[:, :, None, None])
    return x.double()


def _wide_read(st, lens, firsts):
    out = []
    for which in ("k", "v"):
        pool = st[which]
        rows = []
        for r, (ctx, f) in enumerate(zip(lens, firsts)):
            ids = st["bt"][r, f // BLOCK:_blocks(ctx)].long()
            part = {which: pool[ids], which + "_scale": st[which + "_scale"]}
            if pool.dtype == torch.int8:
                part[which + "_exps"] = st[which + "_exps"][ids]
            x = _wide_pool(part, which).transpose(1, 2).reshape(ids.shape[0] * BLOCK, pool.shape[1], pool.shape[3])
            rows.append(x[f - f // BLOCK * BLOCK:ctx - f // BLOCK * BLOCK])
        out.append(torch.cat(rows))
    return out


def _exact_read(case, st):
    s = st["shapes"]
    return tuple(_wide_read(st, s["ctx"], [c - n for c, n in zip(s["ctx"], s["n"])]))


def _exact_write(case, st):
    s = st["shapes"]
    for name in ("k", "v"):
        codes, exps, new = st[name], st[name + "_exps"], st[name + "_new"].double()
        at = 0
        for r, (ctx, n) in enumerate(zip(s["ctx"], s["n"])):
            held = ctx - n
            lo = held // BLOCK
            ids = st["bt"][r, lo:_blocks(ctx)].long()
            nblk = ids.shape[0]
            # New rows on the grid of slots, NaN where there is none.
            grid = torch.full((nblk * BLOCK,) + new.shape[1:], math.nan, dtype=torch.float64, device=DEV)
            grid[held - lo * BLOCK:ctx - lo * BLOCK] = new[at:at + n]
            grid = grid.view(nblk, BLOCK, new.shape[1], new.shape[2]).transpose(1, 2)
            at += n
            top = grid.abs().nan_to_num(nan=0.0).amax((2, 3))
            e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 127.0))
            e = torch.where(top > 127.0 * torch.exp2(e), e + 1.0, e)        # the logarithm may be off at a border
            e = torch.where(top <= 127.0 * torch.exp2(e - 1.0), e - 1.0, e).clamp(min=-126.0)
            old = exps[ids].double()
            keeps = torch.arange(lo, lo + nblk, device=DEV) * BLOCK < held
            e = torch.where(keeps[:, None], torch.maximum(e, old), e)
            unit = torch.exp2(e)[:, :, None, None]
            kept = torch.round(codes[ids].double() * torch.exp2(old - e).clamp(max=1.0)[:, :, None, None])
            codes[ids] = torch.where(grid.isnan(), kept, torch.round(grid / unit)).to(torch.int8)
            exps[ids] = e.to(torch.int8)
    k, v = _wide_read(st, s["ctx"], _touched(s))
    return k, v, st["k_exps"], st["v_exps"]


def _exact_attn(case, st):
    s, g = st["shapes"], case["hq"] // case["hkv"]
    if sum(n * c for n, c in zip(s["n"], s["ctx"])) * case["hq"] * case["d"] * 4 > 6e12:
        return None
    o = torch.zeros((st["q"].shape[0], case["hq"], case["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((st["q"].shape[0], case["hq"]), dtype=torch.float64, device=DEV)
    keys, values = _wide_read(st, s["ctx"], [0] * case["reqs"])
    at = base = 0
    for r, (ctx, n) in enumerate(zip(s["ctx"], s["n"])):
        pos = torch.arange(ctx - n, ctx, device=DEV)
        j = torch.arange(ctx, device=DEV)
        low = torch.zeros_like(pos)
        if case.get("window"):
            low = torch.maximum(low, pos - case["window"] + 1)
        if case.get("docs"):
            low = torch.maximum(low, torch.tensor(s["first"][at:at + n], device=DEV))
        hidden = ((j > pos[:, None]) | (j < low[:, None])) & ~(j < s["prefix"][r])
        for h in range(case["hq"]):
            k, v = keys[base:base + ctx, h // g], values[base:base + ctx, h // g]
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                x = st["q"][at + a:at + b, h].double() @ k.t() * st["scale"]
                if case.get("softcap"):
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if case.get("slopes"):
                    x = x - st["slopes"][h].double() * (pos[a:b, None] - j).abs()
                x = x.masked_fill(hidden[a:b], -math.inf)
                z = torch.logsumexp(x, 1)
                lse[at + a:at + b, h] = z
                o[at + a:at + b, h] = torch.exp(x - z.nan_to_num(neginf=0.0)[:, None]) @ v
        at += n
        base += ctx
    return o, lse


# ---------------------------------------------------------------------------------------------- work
def _seen(case, s):
    """(keys that some token of a request sees, summed; pairs of token and key)."""
    keys = pairs = at = 0
    for r, (ctx, n) in enumerate(zip(s["ctx"], s["n"])):
        pre, lowest = s["prefix"][r], ctx
        for i in range(n):
            p = ctx - n + i
            low = max(pre, p - case["window"] + 1 if case.get("window") else 0, s["first"][at + i] if case.get("docs") else 0)
            pairs += pre + max(0, p + 1 - low)
            lowest = min(lowest, max(pre, low))
        keys += pre + max(0, ctx - lowest)
        at += n
    return keys, pairs


def work(case):
    s = _shapes(case)
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    size = 2 if case["dtype"] == "bf16" else 1
    tokens = sum(s["n"])
    if case["op"] == "attn":
        keys, pairs = _seen(case, s)
        return {"bytes": 2 * hkv * d * size * keys + tokens * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    if case["op"] == "read":
        return {"bytes": 2 * hkv * d * (size + 2) * tokens, "flops": 2 * hkv * d * tokens}
    back = sum(c - f for c, f in zip(s["ctx"], _touched(s)))
    blocks = sum(_blocks(c) - f // BLOCK for c, f in zip(s["ctx"], _touched(s)))
    return {"bytes": 2 * hkv * (d * (3 * tokens + 3 * back) + blocks), "flops": 4 * hkv * d * tokens}
