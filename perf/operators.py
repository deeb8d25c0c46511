"""Work of the serving step over FP8 K/V blocks that carry a scale for each block and kv head.

One step is: block tables and slots of the requests (``build``), the cache write of the new
tokens (``append``), attention of prompts or chunks (``prefill``) or of single tokens
(``decode``) over the cache, and the block copies of copy-on-write (``copy``).  Each case names
one of these operators and its sizes; ``run`` makes one pass through it, in plain torch
operations or, with ``own`` set, through the library.

Cache format: E4M3 codes [blocks][kv heads][block size][head dim] and float32 scales
[blocks][kv heads], K and V apart; a cached value is code * scale.  The write chooses the
smallest power of two 2^e with amax <= 448 * 2^e.
"""
import math
import random

import torch

own = False

LOWEST, HIGHEST = -100, 120  # exponents of the scales that the write stores
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's bookkeeping of 64 chat requests: the smallest call, latency counts
        dict(name="build_decode", op="build", seqs=64, new_lo=1, new_hi=1, past_lo=127, past_hi=2047,
             block=16, mix=1),
        # a ragged wave of prompts and chunks, many of them odd, over an admission burst
        dict(name="build_prompts", op="build", seqs=256, new_lo=1, new_hi=2048, past_lo=0,
             past_hi=1500, block=16, mix=2),
        # the write of one token per request
        dict(name="append_decode", op="append", seqs=64, new_lo=1, new_hi=1, past_lo=127,
             past_hi=2047, heads=8, dim=128, block=16, dtype="bf16", mix=3),
        # prompts of uneven lengths from scratch and chunks that begin inside a block
        dict(name="append_prompts", op="append", seqs=13, new_lo=300, new_hi=2048, past_lo=0,
             past_hi=700, heads=8, dim=128, block=16, dtype="bf16", mix=4),
        # four short sequences, the smallest attention call
        dict(name="decode_tiny", op="decode", seqs=4, past_lo=7, past_hi=100, group=2, heads=2,
             dim=64, block=16, dtype="fp16", mix=5),
        # 64 chat requests of 128..2048 tokens, grouped queries
        dict(name="decode_llama31_8b", op="decode", seqs=64, past_lo=128, past_hi=2048, group=4,
             heads=8, dim=128, block=16, dtype="bf16", mix=6),
        # many short and few long requests, one query head per kv head
        dict(name="decode_mha", op="decode", seqs=128, past_lo=16, past_hi=2048, group=1, heads=32,
             dim=128, block=16, dtype="fp16", mix=7),
        # eight long documents
        dict(name="decode_long", op="decode", seqs=8, past_lo=8192, past_hi=32768, group=4, heads=8,
             dim=128, block=32, dtype="bf16", mix=8),
        # prompts from scratch
        dict(name="prefill_llama31_8b", op="prefill", seqs=8, new_lo=2048, new_hi=2048, past_lo=0,
             past_hi=0, group=4, heads=8, dim=128, block=16, dtype="bf16", mix=9),
        # ragged chunks of longer prompts
        dict(name="prefill_chunked", op="prefill", seqs=16, new_lo=100, new_hi=512, past_lo=1024,
             past_hi=3500, group=4, heads=8, dim=128, block=16, dtype="fp16", mix=10),
        # copy-on-write of two beam searches' last blocks
        dict(name="copy_beam", op="copy", pairs=14, heads=8, dim=128, block=16),
        # whole requests moved within the pool
        dict(name="copy_many", op="copy", pairs=4000, heads=8, dim=128, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["build", "append", "decode", "decode", "prefill", "copy"])
    block = rng.choice([8, 16, 16, 32])
    mix = rng.randrange(1 << 20)
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "build":
        seqs = _log(rng, 1, 1000)
        return dict(op=op, seqs=seqs, new_lo=rng.choice([0, 1]),
                    new_hi=_log(rng, 1, max(1, min(4000, 250000 // seqs))), past_lo=0,
                    past_hi=_log(rng, 1, 4000), block=block, mix=mix)
    if op == "copy":
        return dict(op=op, pairs=_log(rng, 1, 3000), heads=rng.choice([1, 2, 3, 5, 8]), dim=dim,
                    block=block)
    if op == "append":
        seqs, heads = _log(rng, 1, 300), rng.choice([1, 2, 4, 5, 8, 16])
        most = max(1, min(3000, 120000 // (seqs * heads)))
        return dict(op=op, seqs=seqs, new_lo=1, new_hi=_log(rng, 1, most), past_lo=0,
                    past_hi=_log(rng, 1, 600), heads=heads, dim=dim, block=block, dtype=dtype, mix=mix)
    group, heads = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 3, 5, 8, 8, 12])
    if op == "decode":
        seqs = _log(rng, 1, 250)
        most = max(2, min(20000, 200000 * 8 // (seqs * heads * max(1, group // 4))))
        return dict(op=op, seqs=seqs, past_lo=1, past_hi=_log(rng, 2, most), group=group,
                    heads=heads, dim=dim, block=block, dtype=dtype, mix=mix)
    heads = min(heads, 8)
    group = min(group, 8)
    seqs = _log(rng, 1, 16)
    most = max(1, min(1500, 10000 // seqs))
    return dict(op=op, seqs=seqs, new_lo=1, new_hi=_log(rng, 1, most), past_lo=0,
                past_hi=_log(rng, 1, 2500), group=group, heads=heads, dim=dim, block=block,
                dtype=dtype, mix=mix)


def _lengths(case):
    """(new tokens, tokens already cached) of each sequence: part of the case, not of the seed.
    Spread evenly over a narrow range and over the logarithm of a wide one."""
    r = random.Random(case["mix"])

    def one(lo, hi):
        return _log(r, max(lo, 1), hi) if hi > 20 * max(lo, 1) and r.random() < 0.7 else r.randint(lo, hi)

    past = [one(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    new = [one(case["new_lo"], case["new_hi"]) for _ in past] if "new_hi" in case else [0] * len(past)
    return new, past


def work(case):
    op, B = case["op"], case["block"]
    if op == "copy":
        return {"bytes": 2.0 * case["pairs"] * (2 * case["heads"] * B * case["dim"] + 8 * case["heads"]) + 8 * case["pairs"],
                "flops": 0.0}
    new, past = _lengths(case)
    ctx = [a + b for a, b in zip(new, past)]
    used = [-(-c // B) for c in ctx]
    fresh = [u - -(-p // B) for u, p in zip(used, past)]
    if op == "build":
        tables = sum(u - f for u, f, n in zip(used, fresh, new) if n and f < u)
        return {"bytes": 8.0 * len(ctx) + 4.0 * len(ctx) + 8.0 * sum(fresh) + 8.0 * sum(new) + 4.0 * min(tables, len(ctx)),
                "flops": 2.0 * sum(new)}
    H, d = case["heads"], case["dim"]
    if op == "append":
        touched = sum(-(-c // B) - p // B for c, p, n in zip(ctx, past, new) if n)
        return {"bytes": 6.0 * H * d * sum(new) + 8.0 * H * touched + 4.0 * touched,
                "flops": 4.0 * H * d * sum(new)}
    hq = H * case["group"]
    cache = 2.0 * H * d * sum(ctx) + (8.0 * H + 4.0) * sum(used)
    if op == "decode":
        return {"bytes": cache + 4.0 * hq * d * len(ctx), "flops": 4.0 * hq * d * sum(ctx)}
    keys = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return {"bytes": cache + 4.0 * hq * d * sum(new), "flops": 4.0 * hq * d * keys}


# ------------------------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(blocks, case, gen):
    """Codes and scales of one cache: normal values, each (block, head) with a spread of its
    own, as a write of whole blocks leaves them."""
    x = torch.randn(blocks, case["heads"], case["block"], case["dim"], generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-2, 3, (blocks, case["heads"], 1, 1), generator=gen, device="cuda").float())
    s = _scale_of(x.abs().amax(dim=(2, 3)))
    codes = (x / s[:, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["block"]
    st = dict(case)
    if op == "copy":
        blocks = 2 * case["pairs"] + 9
        st["kc"], st["ks"] = _cache(blocks, case, gen)
        st["vc"], st["vs"] = _cache(blocks, case, gen)
        st["pairs"] = torch.randperm(blocks, generator=gen, device="cuda")[:2 * case["pairs"]].view(-1, 2).int().contiguous()
        return st
    new, past = _lengths(case)
    n, ctx = len(new), [a + b for a, b in zip(new, past)]
    used = [-(-c // B) for c in ctx]
    width = max(max(used), 1) + 1
    blocks = sum(used) + max(4, sum(used) // 8)
    order = torch.randperm(blocks, generator=gen, device="cuda").int()
    lens, news = _i32(ctx), _i32(new)
    at = torch.arange(width, device="cuda")[None, :]
    have = _i32([-(-p // B) for p in past] if op == "build" else used)
    start = torch.cumsum(have, 0) - have
    tables = torch.where(at < have[:, None], order[(start[:, None] + at).clamp(max=blocks - 1)], -1).int().contiguous()
    st.update(context_lens=lens, block_tables=tables, blocks=blocks, tokens=sum(new), most=max(new),
              scale=1.0 / math.sqrt(case.get("dim", 64)))
    query_start = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    query_start[1:] = torch.cumsum(news, 0)
    if op == "build":
        # a reserve of free blocks of which the host handed some out before, and a slot buffer
        # of a captured step's fixed size, longer than the tokens of this one
        st["free_blocks"] = order[int(have.sum()):].contiguous()
        st["free_start"] = _i32([min(2, len(st["free_blocks"]) - sum(used) + int(have.sum()))])
        st.update(query_lens=news, slot_mapping=torch.empty(sum(new) + 37, dtype=torch.int64, device="cuda"),
                  query_start=torch.empty(n + 1, dtype=torch.int32, device="cuda"),
                  free_next=torch.empty(1, dtype=torch.int32, device="cuda"))
        return st
    st["query_start"] = query_start
    dt = DTYPES[case["dtype"]]
    st["kc"], st["ks"] = _cache(blocks, case, gen)
    st["vc"], st["vs"] = _cache(blocks, case, gen)
    # rows that no token has been written to hold NaN
    if op == "append":
        full = _i32(past)
    else:
        full = lens
    p = torch.arange(width * B, device="cuda")[None, :]
    ids = tables.clamp(min=0).long().repeat_interleave(B, 1)
    dead = (p >= full[:, None]) & (tables.repeat_interleave(B, 1) >= 0)
    for c in (st["kc"], st["vc"]):
        c.transpose(1, 2)[ids[dead], (p % B).expand(n, -1)[dead]] = 127
    if op == "append":
        shape = (sum(new) + 5, case["heads"], case["dim"])
        gain = torch.exp2(2 * torch.randn(shape[0], shape[1], 1, generator=gen, device="cuda"))
        st["key"] = (torch.randn(shape, generator=gen, device="cuda") * gain).to(dt)
        st["value"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    else:
        rows = n if op == "decode" else sum(new)
        st["q"] = torch.randn(rows, case["heads"] * case["group"], case["dim"], generator=gen, device="cuda").to(dt)
    return st


# ------------------------------------------------------------------------------- plain forms

def _scale_of(amax):
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), LOWEST).clamp(LOWEST, HIGHEST)
    return ((e + 127).int() << 23).view(torch.float32)  # 2^e, exactly


def _codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _build(st):
    B, blocks = st["block"], st["blocks"]
    q, c, tables, free = st["query_lens"].long(), st["context_lens"].long(), st["block_tables"], st["free_blocks"]
    n, width = tables.shape
    total = torch.cumsum(q, 0)
    st["query_start"][0] = 0
    st["query_start"][1:] = total
    have = (c - q + B - 1) // B
    need = (c + B - 1) // B - have
    off = st["free_start"].long() + torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")[None, :]
    fresh = free[(off[:, None] + j - have[:, None]).clamp(0, len(free) - 1)]
    tables.copy_(torch.where((j >= have[:, None]) & (j < (have + need)[:, None]), fresh, tables))
    i = torch.arange(len(st["slot_mapping"]), device="cuda")
    s = torch.searchsorted(total, i, right=True).clamp(max=n - 1)
    p = (c - total)[s] + i
    slot = tables[s, (p // B).clamp(0, width - 1)].long() * B + p % B
    st["slot_mapping"].copy_(torch.where(i < total[-1], slot, -1))
    st["free_next"].copy_(st["free_start"] + need.sum())
    return st["slot_mapping"], tables, st["query_start"], st["free_next"]


def _append(st):
    B, total = st["block"], st["tokens"]
    tables, qs, ctx = st["block_tables"].long(), st["query_start"].long(), st["context_lens"].long()
    n = len(ctx)
    i = torch.arange(total, device="cuda")
    s = torch.searchsorted(qs[1:].contiguous(), i, right=True)
    p = ctx[s] - qs[s + 1] + i
    blk, row = tables[s, p // B], p % B
    lead = (row == 0) | (i == qs[s])
    grp = torch.cumsum(lead, 0) - 1
    new = qs[1:] - qs[:-1]
    first = ((ctx - new) // B).clamp(max=tables.shape[1] - 1)
    r0 = (ctx - new) % B
    fb = tables[torch.arange(n, device="cuda"), torch.minimum(first, (ctx - 1).clamp(min=0) // B)]
    g0 = grp[qs[:-1].clamp(max=max(total - 1, 0))]  # the group of each sequence's first token
    grows = (new > 0) & (r0 > 0)
    for x, codes, scales in ((st["key"], st["kc"], st["ks"]), (st["value"], st["vc"], st["vs"])):
        x = x[:total].float()
        H = x.shape[1]
        amax = torch.zeros(total, H, device="cuda").scatter_reduce_(
            0, grp[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        call = _scale_of(amax)
        old = scales[fb]
        s0 = torch.where(grows[:, None], torch.maximum(old, call[g0]), call[g0])
        block = codes[fb]
        again = _codes(block.view(torch.float8_e4m3fn).float() * (old / s0)[:, :, None, None]).view(torch.uint8)
        earlier = (torch.arange(B, device="cuda")[None, :] < r0[:, None]) & grows[:, None]
        codes[fb] = torch.where(earlier[:, None, :, None], again, block)
        mine = torch.where((grp == g0[s])[:, None], s0[s], call[grp])
        scales[blk] = mine
        codes.transpose(1, 2)[blk, row] = _codes(x / mine[:, :, None]).view(torch.uint8)
    return _append_out(st)


def _append_out(st):
    """The cache as it is held: E4M3 values and the scales that multiply them."""
    f8 = torch.float8_e4m3fn
    return {"k": st["kc"].view(f8), "v": st["vc"].view(f8), "k_scales": st["ks"], "v_scales": st["vs"]}


def _dense(codes, scales, tables, lens):
    """[seqs, heads, width * B, d] float32 values of the tables' blocks, zeros past each length."""
    n, width = tables.shape
    ids = tables.clamp(min=0).long()
    x = codes[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]  # n, T, H, B, d
    x = x.transpose(1, 2).reshape(n, codes.shape[1], -1, codes.shape[3])
    live = torch.arange(x.shape[2], device="cuda")[None, :] < lens[:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def _attend(q, k, v, live, scale):
    """q [n, H, rows, d], live [n, 1 or H, rows or 1, L]."""
    z = torch.matmul(q, k.transpose(2, 3)) * scale
    z = torch.where(live, z, -torch.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _decode(st):
    k, live = _dense(st["kc"], st["ks"], st["block_tables"], st["context_lens"])
    v, _ = _dense(st["vc"], st["vs"], st["block_tables"], st["context_lens"])
    q = st["q"]
    n, hq, d = q.shape
    o = _attend(q.float().view(n, st["heads"], -1, d), k, v, live[:, None, None, :], st["scale"])
    return o.reshape(n, hq, d).to(q.dtype)


def _prefill(st):
    k, live = _dense(st["kc"], st["ks"], st["block_tables"], st["context_lens"])
    v, _ = _dense(st["vc"], st["vs"], st["block_tables"], st["context_lens"])
    q, qs, ctx = st["q"], st["query_start"].long(), st["context_lens"].long()
    N, hq, d = q.shape
    n, H, G, most = len(ctx), st["heads"], st["group"], st["most"]
    j = torch.arange(most, device="cuda")[None, :]
    x = q.float()[(qs[:-1, None] + j).clamp(max=N - 1)].view(n, most, H, G, d)
    x = x.permute(0, 2, 3, 1, 4).reshape(n, H, G * most, d)
    pos = (ctx - qs[1:] + qs[:-1])[:, None] + j  # position of each query
    see = (torch.arange(k.shape[2], device="cuda")[None, None, :] <= pos[:, :, None]) & live[:, None, :]
    o = _attend(x, k, v, see.repeat(1, G, 1)[:, None], st["scale"]).view(n, H, G, most, d)
    i = torch.arange(N, device="cuda")
    s = torch.searchsorted(qs[1:].contiguous(), i, right=True)
    return o.permute(0, 3, 1, 2, 4)[s, i - qs[s]].reshape(N, hq, d).to(q.dtype)


def _copy(st):
    src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    for t in (st["kc"], st["vc"], st["ks"], st["vs"]):
        t[dst] = t[src]
    return _append_out(st)


# ------------------------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        import paged_kv_cache_149_gb300 as pa
        if op == "build":
            pa.build_step(st["query_lens"], st["context_lens"], st["free_blocks"], st["free_start"],
                          st["block_tables"], st["block"], st["blocks"], st["slot_mapping"],
                          st["query_start"], st["free_next"])
            return st["slot_mapping"], st["block_tables"], st["query_start"], st["free_next"]
        cache = (st["kc"], st["vc"], st["ks"], st["vs"])
        if op == "append":
            pa.append_fp8_block(st["key"], st["value"], *cache, st["block_tables"],
                                st["context_lens"], st["query_start"])
            return _append_out(st)
        if op == "copy":
            pa.copy_blocks_fp8_block(*cache, st["pairs"])
            return _append_out(st)
        if op == "decode":
            if "workspace" not in st:  # a serving loop keeps its workspace from step to step
                st["workspace"] = pa.make_workspace(st["q"].shape[1], st["heads"], st["dim"])
            return pa.decode_fp8_block(st["q"], *cache, st["block_tables"], st["context_lens"],
                                       st["scale"], workspace=st["workspace"])
        return pa.prefill_fp8_block(st["q"], *cache, st["block_tables"], st["context_lens"],
                                    st["query_start"], st["scale"], st["most"])
    return {"build": _build, "append": _append, "decode": _decode, "prefill": _prefill, "copy": _copy}[op](st)


# ------------------------------------------------------------------------------- in 64 bits

def _value_table():
    """The 256 values of E4M3 codes, from the format's definition."""
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        t.append(-v if c & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """float64 values to the nearest E4M3 value, ties to even, magnitudes above 448 to 448."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    op, B = case["op"], case["block"]
    if op == "build":
        return None
    st = prepare(case, seed)
    value = _value_table()
    if op == "copy":
        out = {"k": value[st["kc"].long()], "v": value[st["vc"].long()], "k_scales": st["ks"].double(), "v_scales": st["vs"].double()}
        src, dst = st["pairs"].long().T
        return {name: t.index_copy(0, dst, t[src]) for name, t in out.items()}
    new, past = _lengths(case)
    tables, begin = st["block_tables"].tolist(), 0
    if op == "append":
        out = {"k": value[st["kc"].long()], "v": value[st["vc"].long()], "k_scales": st["ks"].double(), "v_scales": st["vs"].double()}
        for s, (n, p) in enumerate(zip(new, past)):
            for j in range(p // B, -(-(p + n) // B)):
                lo, hi = max(p, j * B), min(p + n, (j + 1) * B)  # positions that this call writes
                b, a, z = tables[s][j], lo - j * B, hi - j * B
                for name, x in (("k", st["key"]), ("v", st["value"])):
                    rows = x[begin + lo - p:begin + hi - p].double().transpose(0, 1)
                    big = rows.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(big / 448))
                    e = torch.where(448 * torch.exp2(e - 1) >= big, e - 1, e)  # (a log2 rounded up)
                    scale = torch.exp2(e.clamp(LOWEST, HIGHEST))
                    if a:
                        was = out[name + "_scales"][b]
                        scale = torch.maximum(scale, was)
                        out[name][b, :, :a] = _round_e4m3(out[name][b, :, :a] * (was / scale)[:, None, None])
                    out[name + "_scales"][b] = scale
                    out[name][b, :, a:z] = _round_e4m3(rows / scale[:, None, None])
            begin += n
        return out
    q = st["q"].double()
    out = torch.zeros_like(q)
    for s, (n, p) in enumerate(zip(new, past)):
        c = n + p
        ids = torch.tensor(tables[s][:-(-c // B)], device="cuda")
        k, v = ((value[codes[ids].long()] * scales[ids].double()[:, :, None, None]).transpose(1, 2).reshape(-1, case["heads"], case["dim"])[:c]
                for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        rows = q[s:s + 1] if op == "decode" else q[begin:begin + n]
        first = c - len(rows)
        for h in range(case["heads"]):
            heads = slice(h * case["group"], (h + 1) * case["group"])
            z = torch.einsum("rgd,td->grt", rows[:, heads], k[:, h]) * st["scale"]
            late = torch.arange(c, device="cuda")[None, :] > first + torch.arange(len(rows), device="cuda")[:, None]
            w = torch.softmax(z.masked_fill(late, -math.inf), -1)
            got = torch.einsum("grt,td->rgd", w, v[:, h])
            if op == "decode":
                out[s, heads] = got[0]
            else:
                out[begin:begin + n, heads] = got
        begin += n
    return out
