"""Work of a decoding step that checks drafted tokens, and of attention to an encoder's states.

A step feeds each sequence its last token and some drafted ones.  ``rotary`` turns the new
queries and keys by their positions and writes the new K/V rows into the paged cache;
``drafts`` is the causal attention of those few tokens over the sequence's long context;
``cross`` attends from any number of tokens to states of another length that lie in the same
kind of blocks, without a mask; ``verify`` accepts or rejects the drafts against the target's
probabilities, from given random numbers, and samples the token after them.  Each case names
one of these operators and its sizes; ``run`` makes one pass through it, in plain torch
operations or, with ``own`` set, through the library.

Caches are fp16 or bf16 [blocks][kv heads][block size][head dim], K and V apart.  Sequence s owns
rows query_start[s] .. query_start[s + 1] - 1 of the step's tensors; rows behind the last
sequence (a padded batch) belong to none.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of each of 64 chat requests: the smallest call, latency counts
        dict(name="rotary_decode", op="rotary", seqs=64, new_lo=1, new_hi=1, past_lo=127, past_hi=2047,
             group=4, heads=8, dim=128, block=16, dtype="bf16", rotary=128, pairs="half",
             scaling="none", fused=True, mix=1),
        # drafted tokens of many requests, one query head per kv head, half of each head turned
        dict(name="rotary_drafts", op="rotary", seqs=256, new_lo=1, new_hi=8, past_lo=16, past_hi=4000,
             group=1, heads=32, dim=128, block=16, dtype="fp16", rotary=64, pairs="interleaved",
             scaling="none", fused=True, mix=2),
        # prompts and chunks that begin inside a block, far into a context stretched past its training
        dict(name="rotary_prompts", op="rotary", seqs=13, new_lo=300, new_hi=2048, past_lo=0,
             past_hi=100000, group=4, heads=8, dim=128, block=16, dtype="bf16", rotary=128, pairs="half",
             scaling="bands", fused=False, mix=3),
        # four short sequences, the smallest attention call
        dict(name="drafts_tiny", op="drafts", seqs=4, new_lo=1, new_hi=4, past_lo=7, past_hi=100,
             group=2, heads=2, dim=64, block=16, dtype="fp16", mix=4),
        # 64 chat requests with up to seven drafted tokens each
        dict(name="drafts_llama31_8b", op="drafts", seqs=64, new_lo=1, new_hi=8, past_lo=128,
             past_hi=2048, group=4, heads=8, dim=128, block=16, dtype="bf16", mix=5),
        # eight long documents, a drafted continuation of each
        dict(name="drafts_long", op="drafts", seqs=8, new_lo=5, new_hi=16, past_lo=8192, past_hi=32768,
             group=4, heads=8, dim=128, block=32, dtype="bf16", mix=6),
        # one decoder token of each of 64 requests to its encoder's states
        dict(name="cross_step", op="cross", seqs=64, new_lo=1, new_hi=1, past_lo=100, past_hi=1500,
             group=1, heads=16, dim=64, block=16, dtype="fp16", mix=7),
        # the decoder's prompts of uneven lengths
        dict(name="cross_prompts", op="cross", seqs=32, new_lo=3, new_hi=448, past_lo=100, past_hi=1500,
             group=1, heads=16, dim=64, block=16, dtype="fp16", mix=8),
        # long texts against long documents, grouped queries
        dict(name="cross_long", op="cross", seqs=6, new_lo=900, new_hi=2048, past_lo=2000, past_hi=8192,
             group=4, heads=8, dim=128, block=32, dtype="bf16", mix=9),
        # four requests, three drafts each
        dict(name="verify_small", op="verify", seqs=4, new_lo=4, new_hi=4, past_lo=10, past_hi=100,
             vocab=32000, dtype="fp32", drawn=True, accept=70, mix=10),
        # a batch of chat requests with up to seven drafts each
        dict(name="verify_chat", op="verify", seqs=64, new_lo=1, new_hi=8, past_lo=128, past_hi=2048,
             vocab=128256, dtype="fp32", drawn=True, accept=75, mix=11),
        # drafts looked up in the text, with no probabilities of their own; an odd vocabulary
        dict(name="verify_lookup", op="verify", seqs=192, new_lo=1, new_hi=6, past_lo=16, past_hi=4000,
             vocab=50257, dtype="bf16", drawn=False, accept=60, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "drafts", "drafts", "cross", "cross", "verify"])
    mix = rng.randrange(1 << 20)
    if op == "verify":
        seqs, vocab = _log(rng, 1, 250), _log(rng, 1000, 150000)
        most = max(1, min(12, 40000000 // (seqs * vocab)))
        return dict(op=op, seqs=seqs, new_lo=rng.choice([0, 1, 1]), new_hi=rng.randint(1, most),
                    past_lo=0, past_hi=3000, vocab=vocab, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    drawn=rng.random() < 0.7, accept=rng.choice([0, 50, 75, 100]), mix=mix)
    dim = rng.choice([64, 128, 128])
    case = dict(op=op, dim=dim, block=rng.choice([8, 16, 16, 32]), dtype=rng.choice(["bf16", "fp16"]),
                group=rng.choice([1, 2, 3, 4, 7, 8, 16]), heads=rng.choice([1, 2, 3, 5, 8, 8, 16]), mix=mix)
    wide = case["heads"] * case["group"]
    if op == "rotary":
        seqs = _log(rng, 1, 300)
        most = max(1, min(2500, 500000 // (seqs * wide)))
        case.update(seqs=seqs, new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, most), past_lo=0,
                    past_hi=_log(rng, 1, 20000), rotary=16 * rng.randint(1, dim // 16),
                    pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "bands", "ramp"]), fused=rng.random() < 0.5)
        return case
    if op == "drafts":
        seqs = _log(rng, 1, 200)
        most = max(2, min(30000, 1500000 // (seqs * case["heads"])))
        case.update(seqs=seqs, new_lo=1, new_hi=_log(rng, 1, max(1, min(40, 20000 // (seqs * wide)))),
                    past_lo=0, past_hi=_log(rng, 2, most))
        return case
    seqs = _log(rng, 1, 100)
    case.update(seqs=seqs, new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, max(1, min(1500, 60000 // (seqs * wide)))),
                past_lo=rng.choice([0, 1]), past_hi=_log(rng, 1, max(2, min(8000, 800000 // (seqs * case["heads"])))))
    return case


def _lengths(case):
    """(new tokens, tokens already cached) of each sequence: part of the case, not of the seed.
    Spread evenly over a narrow range and over the logarithm of a wide one.  For attention to an
    encoder the second is the number of its states."""
    r = random.Random(case["mix"])

    def one(lo, hi):
        return _log(r, max(lo, 1), hi) if hi > 20 * max(lo, 1) and r.random() < 0.7 else r.randint(lo, hi)

    past = [one(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    new = [one(case["new_lo"], case["new_hi"]) for _ in past]
    return new, past


def _taken(case, new):
    """Drafts accepted of each sequence (of its new tokens, all but the first)."""
    r = random.Random(case["mix"] + 1)
    out = []
    for n in new:
        k = 0
        while k < n - 1 and r.randrange(100) < case["accept"]:
            k += 1
        out.append(k)
    return out


def work(case):
    new, past = _lengths(case)
    if case["op"] == "verify":
        took, size = _taken(case, new), DTYPES[case["dtype"]].itemsize
        rows = sum((2 if case["drawn"] and k < n - 1 else 1) for n, k in zip(new, took) if n)
        looks = sum(min(k + 1, n - 1) for n, k in zip(new, took) if n)
        return {"bytes": float(rows * case["vocab"] * size + looks * (8 + 2 * size) + 4 * sum(new) + 20 * len(new)),
                "flops": 2.0 * rows * case["vocab"]}
    H, G, d, B = case["heads"], case["group"], case["dim"], case["block"]
    if case["op"] == "rotary":
        rows = sum(new)
        tables = sum(-(-(p + n) // B) - p // B for n, p in zip(new, past) if n)
        return {"bytes": 4.0 * rows * d * H * (G + 2) + 4.0 * tables + 8.0 * len(new),
                "flops": 3.0 * rows * case["rotary"] * H * (G + 1)}
    ctx = [p + n for n, p in zip(new, past)] if case["op"] == "drafts" else past
    cache = sum(4.0 * H * d * c + 4.0 * -(-c // B) for c, n in zip(ctx, new) if n)
    if case["op"] == "drafts":
        keys = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    else:
        keys = sum(n * c for n, c in zip(new, ctx))
    return {"bytes": cache + 4.0 * H * G * d * sum(new) + 8.0 * len(new), "flops": 4.0 * H * G * d * keys}


# ------------------------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


SCALING = {  # how the angles of long contexts are stretched, as a user names it
    "none": None,
    "linear": dict(kind="linear", factor=4.0),
    "bands": dict(kind="bands", factor=8.0, low=1.0, high=4.0, trained=8192),
    "ramp": dict(kind="ramp", factor=16.0, slow=1.0, fast=32.0, trained=4096),
}
BASE = 500000.0


def _angles_per_token(case):
    """float64 radians per token of each pair, and the factor on cosines and sines.
    linear: f / factor.  bands: f where the trained length holds more than `high` turns, f / factor
    where fewer than `low`, between them blended by the number of turns.  ramp: f / factor and f
    blended linearly in the pair's index between the (whole) indexes whose pairs make `fast` and
    `slow` turns over the trained length, and amplitudes 0.1 ln(factor) + 1."""
    rd, how = case["rotary"], SCALING[case["scaling"]]
    f = [BASE ** (-2.0 * i / rd) for i in range(rd // 2)]
    amplitude = 1.0
    if how and how["kind"] == "linear":
        f = [x / how["factor"] for x in f]
    elif how and how["kind"] == "bands":
        out = []
        for x in f:
            turns = how["trained"] * x / (2 * math.pi)
            a = min(1.0, max(0.0, (turns - how["low"]) / (how["high"] - how["low"])))
            out.append((1 - a) * x / how["factor"] + a * x)
        f = out
    elif how:
        def index(turns):
            return rd * math.log(how["trained"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo = max(math.floor(index(how["fast"])), 0)
        hi = min(math.ceil(index(how["slow"])), rd - 1)
        out = []
        for i, x in enumerate(f):
            a = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(a * x / how["factor"] + (1 - a) * x)
        f = out
        amplitude = 0.1 * math.log(how["factor"]) + 1.0
    return f, amplitude


def _verify_inputs(case, st, gen):
    """Probabilities of two models that mostly agree, and drafts and random numbers that lead to
    the case's counts of accepted drafts: a draft that will be refused is drawn from what the
    draft model has too much of, its random number lies above the ratio of the two."""
    new, _ = _lengths(case)
    N, V = sum(new), case["vocab"]
    dt = DTYPES[case["dtype"]]
    z = 3 * torch.randn(N + 3, V, generator=gen, device="cuda")
    p = torch.softmax(z, -1).to(dt)
    z += 0.7 * torch.randn(N + 3, V, generator=gen, device="cuda")
    q = torch.softmax(z, -1).to(dt)
    del z
    took, refuse, first, at = _taken(case, new), [], [], 0
    for n, k in zip(new, took):
        if n:
            first.append(at)
            if k < n - 1:
                refuse.append(at + k)
        at += n
    N2 = p.shape[0]
    no = torch.zeros(N2, dtype=torch.bool, device="cuda")
    no[torch.tensor(refuse, dtype=torch.long, device="cuda")] = True
    u = torch.rand(N2, generator=gen, device="cuda")
    token = torch.randint(0, V, (N2,), generator=gen, device="cuda")  # first tokens, padding
    for a in range(0, max(N - 1, 0), 64):  # draft r + 1 is judged by row r
        b = min(a + 64, N - 1)
        pa, qa, bad = p[a:b].float(), q[a:b].float(), no[a:b]
        if case["drawn"]:
            w = torch.where(bad[:, None], (qa - pa).clamp(min=0), qa)
            t = torch.multinomial(w, 1, generator=gen)[:, 0]
            ratio = (pa.gather(1, t[:, None])[:, 0] / qa.gather(1, t[:, None])[:, 0]).clamp(max=1)
        else:
            t = torch.multinomial(pa, 1, generator=gen)[:, 0]
            ratio = pa.gather(1, t[:, None])[:, 0]
        token[a + 1:b + 1] = t
        u[a:b] = torch.where(bad, ratio + (1 - ratio) * u[a:b], ratio * u[a:b])
    at = 0
    ends = []
    for n in new:
        at += n
        ends.append(at - 1)
    ends = torch.tensor([e for e, n in zip(ends, new) if n], dtype=torch.long, device="cuda")
    u[ends] = torch.rand(len(ends), generator=gen, device="cuda")  # the sampled token's number
    heads = torch.tensor(first, dtype=torch.long, device="cuda")
    token[heads] = torch.randint(0, V, (len(first),), generator=gen, device="cuda")
    st.update(target=p, draft=q if case["drawn"] else None, step_tokens=token.int(),
              uniforms=u.clamp(max=1 - 2.0 ** -24))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    new, past = _lengths(case)
    n, op = len(new), case["op"]
    ctx = past if op == "cross" else [a + b for a, b in zip(new, past)]
    lens, news = _i32(ctx), _i32(new)
    query_start = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    query_start[1:] = torch.cumsum(news, 0)
    st.update(context_lens=lens, query_start=query_start, tokens=sum(new), most=max(new),
              longest=max(ctx), new=new)
    if op == "verify":
        _verify_inputs(case, st, gen)
        return st
    B, H, G, d, dt = case["block"], case["heads"], case["group"], case["dim"], DTYPES[case["dtype"]]
    width = max(-(-max(ctx) // B), 1) + 1
    used = [-(-c // B) for c in ctx]
    if op == "rotary":  # only the blocks that are written need to exist: earlier entries are not read
        first = [p // B for p in past]
    else:
        first = [0] * n
    blocks = sum(u - f for u, f in zip(used, first)) + 5
    order = torch.randperm(blocks, generator=gen, device="cuda").int()
    at = torch.arange(width, device="cuda")[None, :]
    lo, hi = _i32(first), _i32(used)
    start = torch.cumsum(hi - lo, 0) - (hi - lo)
    mine = (at >= lo[:, None]) & (at < hi[:, None])
    st["block_tables"] = torch.where(mine, order[(start[:, None] + at - lo[:, None]).clamp(0, blocks - 1)], -1).int().contiguous()
    shape = (blocks, H, B, d)
    st["k_cache"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)
    st["v_cache"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)
    rows, Hq = sum(new) + 3, H * G
    if op == "rotary":
        if case["fused"]:  # one projection's output, cut into q, k and v
            x = torch.randn(rows, (Hq + 2 * H) * d, generator=gen, device="cuda").to(dt)
            q, k, v = x.split([Hq * d, H * d, H * d], 1)
        else:
            q, k, v = (torch.randn(rows, h * d, generator=gen, device="cuda").to(dt) for h in (Hq, H, H))
        st.update(q=q.unflatten(1, (Hq, d)), key=k.unflatten(1, (H, d)), value=v.unflatten(1, (H, d)))
        f, st["amplitude"] = _angles_per_token(case)
        st["angles"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        return st
    st["scale"] = 1.0 / math.sqrt(d)
    # rows that no token has been written to hold NaN
    p = torch.arange(width * B, device="cuda")[None, :]
    table = st["block_tables"].long().repeat_interleave(B, 1)
    dead = (p >= lens[:, None]) & (table >= 0)
    for c in (st["k_cache"], st["v_cache"]):
        c.transpose(1, 2)[table[dead], (p % B).expand(n, -1)[dead]] = math.nan
    st["q"] = torch.randn(sum(new), Hq, d, generator=gen, device="cuda").to(dt)
    return st


# ------------------------------------------------------------------------------- plain forms

def _owner(st):
    """(sequence, position) of each of the step's rows."""
    qs, ctx = st["query_start"].long(), st["context_lens"].long()
    i = torch.arange(st["tokens"], device="cuda")
    s = torch.searchsorted(qs[1:].contiguous(), i, right=True)
    return s, ctx[s] - qs[s + 1] + i


def _rotary(st):
    N, rd, B = st["tokens"], st["rotary"], st["block"]
    s, pos = _owner(st)
    turn = pos.double()[:, None] * st["angles"]
    cos, sin = ((f(turn) * st["amplitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))

    def turned(x):
        out = x[:N].float()
        r = out[..., :rd]
        if st["pairs"] == "half":
            a, b = r[..., :rd // 2], r[..., rd // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([r, out[..., rd:]], -1).to(x.dtype)

    blk, row = st["block_tables"][s, pos // B].long(), pos % B
    st["k_cache"].transpose(1, 2)[blk, row] = turned(st["key"])
    st["v_cache"].transpose(1, 2)[blk, row] = st["value"][:N]
    return turned(st["q"]), st["k_cache"], st["v_cache"]


def _attend(st):
    """Sequence after sequence, query heads of a kv head together, in pieces of queries."""
    q, qs, B = st["q"], st["query_start"].tolist(), st["block"]
    ctx, H, d = st["context_lens"].tolist(), st["heads"], st["dim"]
    out = torch.zeros_like(q)
    for s, c in enumerate(ctx):
        a, b = qs[s], qs[s + 1]
        if a == b or c == 0:
            continue
        ids = st["block_tables"][s, :-(-c // B)].long()
        k, v = (st[x][ids].transpose(0, 1).reshape(H, -1, d)[:, :c].float() for x in ("k_cache", "v_cache"))
        step = max(1, (1 << 28) // (c * q.shape[1]))
        for i in range(a, b, step):
            e = min(b, i + step)
            x = q[i:e].float().view(e - i, H, -1, d).permute(1, 2, 0, 3)  # H, G, rows, d
            z = torch.matmul(x, k[:, None].transpose(2, 3)) * st["scale"]
            if st["op"] == "drafts":
                pos = c - b + torch.arange(i, e, device="cuda")
                z = torch.where(torch.arange(c, device="cuda")[None, :] <= pos[:, None], z, -torch.inf)
            w = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(w, v[:, None]) / w.sum(-1, keepdim=True)
            out[i:e] = o.permute(2, 0, 1, 3).reshape(e - i, -1, d).to(q.dtype)
    return out


def _verify(st):
    qs, N, V = st["query_start"].long(), st["tokens"], st["vocab"]
    p, q, u, token = st["target"], st["draft"], st["uniforms"], st["step_tokens"].long()
    n, new = len(qs) - 1, qs[1:] - qs[:-1]
    out = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    j = torch.arange(max(st["most"] - 1, 1), device="cuda")[None, :]
    r = (qs[:-1, None] + j).clamp(max=max(N - 1, 0))
    t = token[(r + 1).clamp(max=len(token) - 1)]
    chance = q[r, t].double() if q is not None else 1.0
    good = (u[r].double() * chance < p[r, t].double()) & (j < new[:, None] - 1)
    took = torch.cumprod(good.long(), 1).sum(1)  # accepted drafts
    row = (qs[:-1] + took).clamp(max=max(N - 1, 0))
    full = p[row].double()
    over = full
    if q is not None:
        over = (full - q[row].double()).clamp(min=0)
    else:
        said = token[(row + 1).clamp(max=len(token) - 1)]
        over = full.scatter(1, said[:, None], 0.0)
    refused = took < new - 1
    w = torch.where(refused[:, None] & (over.sum(1) > 0)[:, None], over, full)
    c = torch.cumsum(w, 1)
    pick = (c <= (u[(qs[1:] - 1).clamp(min=0)].double() * c[:, -1])[:, None]).sum(1)
    live = new > 0
    emitted = torch.where(live, took + 1, 0)
    i = torch.arange(N, device="cuda")
    s = torch.searchsorted(qs[1:].contiguous(), i, right=True)
    k = i - qs[s]
    nxt = token[(i + 1).clamp(max=len(token) - 1)]
    out = torch.where(k < took[s], nxt, torch.where(k == took[s], pick[s], -1)).int()
    left = st["context_lens"].long() - new + emitted
    return out, emitted.int(), left.int()


# ------------------------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        import paged_kv_cache_149_gb300 as pa
        if op == "verify":
            out, emitted, left = pa.verify_drafts(st["step_tokens"], st["target"], st["draft"], st["uniforms"],
                                                  st["query_start"], st["context_lens"])
            return out[:st["tokens"]], emitted, left
        cache = (st["k_cache"], st["v_cache"], st["block_tables"], st["context_lens"], st["query_start"])
        if op == "rotary":
            if "freqs" not in st:  # laid out once for a model
                st["freqs"], st["factor"] = pa.rotary_frequencies(st["rotary"], BASE, SCALING[st["scaling"]])
            out = pa.rotary_append(st["q"], st["key"], st["value"], *cache, st["freqs"],
                                   interleaved=st["pairs"] == "interleaved", amplitude=st["factor"])
            return out[:st["tokens"]], st["k_cache"], st["v_cache"]
        if "workspace" not in st:  # a serving loop keeps its workspace from step to step
            st["workspace"] = pa.make_split_workspace(st["q"].shape[1], st["heads"], st["dim"])
        call = pa.decode_drafts if op == "drafts" else pa.cross
        return call(st["q"], *cache, st["scale"], workspace=st["workspace"])
    return {"rotary": _rotary, "drafts": _attend, "cross": _attend, "verify": _verify}[op](st)


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "verify":  # whole numbers
        return None
    st = prepare(case, seed)
    new, past = _lengths(case)
    tables, B, d = st["block_tables"].tolist(), case["block"], case["dim"]
    begin = 0
    if op == "rotary":
        rd = case["rotary"]
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        q = st["q"][:sum(new)].double()
        f, amplitude = _angles_per_token(case)
        f = torch.tensor(f, dtype=torch.float64, device="cuda")
        for s, (n, p) in enumerate(zip(new, past)):
            if not n:
                continue
            pos = torch.arange(p, p + n, device="cuda", dtype=torch.float64)
            turn = torch.polar(torch.full((n, rd // 2), amplitude, dtype=torch.float64, device="cuda"),
                               pos[:, None] * f[None, :])[:, None, :]
            rows = slice(begin, begin + n)
            k = st["key"][rows].double()
            for x in (q[rows], k):
                part = x[..., :rd].clone()
                if case["pairs"] == "half":
                    z = torch.complex(part[..., :rd // 2], part[..., rd // 2:]) * turn
                    x[..., :rd // 2], x[..., rd // 2:rd] = z.real, z.imag
                else:
                    z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn
                    x[..., :rd] = torch.view_as_real(z).flatten(-2)
            for j in range(p // B, -(-(p + n) // B)):
                lo, hi = max(p, j * B), min(p + n, (j + 1) * B)
                to = slice(lo - j * B, hi - j * B)
                kc[tables[s][j], :, to] = k[lo - p:hi - p].transpose(0, 1)
                vc[tables[s][j], :, to] = st["value"][begin + lo - p:begin + hi - p].double().transpose(0, 1)
            begin += n
        return q, kc, vc
    if work(case)["flops"] > 4e12:
        return None
    q = st["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for s, (n, p) in enumerate(zip(new, past)):
        c = p if op == "cross" else p + n
        if n and c:
            ids = torch.tensor(tables[s][:-(-c // B)], device="cuda")
            for h in range(case["heads"]):
                k, v = (st[x][ids, h].double().reshape(-1, d)[:c] for x in ("k_cache", "v_cache"))
                for g in range(h * case["group"], (h + 1) * case["group"]):
                    z = q[begin:begin + n, g].double() @ k.T * st["scale"]
                    if op == "drafts":
                        z += torch.full_like(z, -math.inf).triu(c - n + 1)
                    out[begin:begin + n, g] = torch.softmax(z, -1) @ v
        begin += n
    return out
