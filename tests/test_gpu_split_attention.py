"""decode_drafts and cross against plain attention in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import DT, Paged, attend64, attention_tolerance, i32, run, starts

pytestmark = pytest.mark.gpu

# lengths that end and begin inside, at and past 64-key tiles and blocks, with few and many rows
CTX = [1, 7, 63, 64, 65, 100, 128, 129, 300, 517, 1000, 2048]
ROWS = [1, 5, 3, 64, 2, 100, 33, 129, 1, 260, 4, 17]
SHAPES = [  # dtype, d, block, query heads per kv head, kv heads
    ("bf16", 128, 16, 4, 2), ("fp16", 64, 8, 1, 3), ("bf16", 64, 32, 7, 1), ("fp16", 128, 32, 16, 1),
    ("bf16", 128, 8, 3, 2), ("fp16", 64, 16, 128, 1), ("bf16", 64, 16, 2, 5), ("fp16", 128, 16, 5, 2),
]


def compare(out, p, q, qs, ctx, scale, causal):
    assert not out[:qs[-1]].isnan().any()
    for s, c in enumerate(ctx):
        a, b = qs[s], qs[s + 1]
        if a == b:
            continue
        ref, mass = attend64(q[a:b], p.k[s], p.v[s], scale, c - (b - a) if causal else None)
        err = (out[a:b].double() - ref).abs()
        assert (err <= attention_tolerance(ref, mass, p.dt, p.d)).all(), (s, c, float(err.max()))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("few", [True, False])
def test_against_64_bits(shape, causal, few):
    dtype, d, block, G, hkv = shape
    rows = [min(r, 3) for r in ROWS] if few else list(ROWS)
    if causal:
        rows = [min(r, c) for r, c in zip(rows, CTX)]
    rows[4] = 0  # a sequence without rows
    qs = starts(rows)
    p = Paged(CTX, hkv, d, block, dtype, seed=len(rows) + d + G)
    q = p.q(qs[-1] + 3, G * hkv)
    scale = 1 / math.sqrt(d)
    out = torch.full_like(q, 7.0).cuda()  # rows behind the last sequence stay as they are
    out, err = run(pa.decode_drafts if causal else pa.cross, p, q, qs, CTX, scale, out=out)
    assert err == 0
    assert (out[qs[-1]:] == 7.0).all()
    compare(out, p, q, qs, CTX, scale, causal)


@pytest.mark.parametrize("ctx,rows", [([5000], [3]), ([1], [1]), ([9000, 40, 1], [2, 40, 1]),
                                      ([20000, 700, 700, 700], [16, 1, 5, 8]), ([513] * 9, [1] * 9),
                                      ([4096] * 3, [200, 1, 130]), ([130] * 200, [1] * 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_and_ragged_batches(ctx, rows, causal):
    p = Paged(ctx, 2, 128, 16, "bf16", seed=3)
    qs = starts(rows)
    q = p.q(qs[-1], 8)
    out, err = run(pa.decode_drafts if causal else pa.cross, p, q, qs, ctx, 0.09)
    assert err == 0
    compare(out, p, q, qs, ctx, 0.09, causal)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_peaked_and_growing_scores(dtype):
    """Scores of hundreds, whose running maximum grows from tile to tile (O is rescaled), cut in
    pieces with very different maxima."""
    ctx, rows = [3000, 700], [4, 9]
    p = Paged(ctx, 1, 64, 16, dtype, seed=5, spread=1.0)
    for k in p.k:  # larger and larger keys
        k.mul_(torch.linspace(0.1, 12, len(k))[:, None, None].to(k.dtype))
    qs = starts(rows)
    q = p.q(qs[-1], 4)
    for causal in (True, False):
        out, err = run(pa.decode_drafts if causal else pa.cross, p, q, qs, ctx, 1.0)
        assert err == 0
        for s, c in enumerate(ctx):
            a, b = qs[s], qs[s + 1]
            ref, mass = attend64(q[a:b], p.k[s], p.v[s], 1.0, c - (b - a) if causal else None)
            # scores of size 400: an addition of the sum of 64 products is off by 2^-23 of up to 1000,
            # so weights by 64 * 1000 * 2^-23 at most
            tol = attention_tolerance(ref, mass, p.dt, 64) + 2 * 64 * 1000 * 2.0 ** -23 * mass
            assert ((out[a:b].double() - ref).abs() <= tol).all()


def test_largest_values_of_f16_stay_finite():
    ctx, rows = [1500], [3]
    p = Paged(ctx, 1, 64, 16, "fp16", seed=6)
    p.v[0].fill_(65504.0)
    p.v[0][:, :, 32:] = -65504.0
    q = p.q(3, 2)
    for call in (pa.decode_drafts, pa.cross):
        out, err = run(call, p, q, [0, 3], ctx, 0.1)
        # (weights rounded by half a step each: an average of equal values is off by one step)
        assert err == 0 and out.isfinite().all()
        assert ((out.double() - p.v[0][0].double()).abs() <= 64).all()


@pytest.mark.parametrize("ctx,rows", [([40], [9]), ([3000], [9]), ([700, 90], [200, 60])])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_keys_not_attended_change_no_bit(ctx, rows, bad, dtype):
    """Later drafts' K/V that is not finite: the rows before keep their bits, the others get it."""
    p = Paged(ctx, 2, 64, 16, dtype, seed=8)
    qs = starts(rows)
    q = p.q(qs[-1], 4)
    clean, err = run(pa.decode_drafts, p, q, qs, ctx, 0.125)
    assert err == 0
    at = [c - r + r // 2 for c, r in zip(ctx, rows)]  # this token's rows are not finite
    for s, t in enumerate(at):
        p.v[s][t, 1, 5] = bad
        p.v[s][t, 1, 40] = bad
        p.k[s][t, 0, 3] = math.nan
    out, err = run(pa.decode_drafts, p, q, qs, ctx, 0.125)
    assert err == 0
    for s, t in enumerate(at):
        cut = qs[s] + t - (ctx[s] - rows[s])
        a, b = qs[s], qs[s + 1]
        assert torch.equal(out[a:cut], clean[a:cut])
        assert out[cut:b, :2].isnan().all()  # K of kv head 0: heads 0 and 1
        late = out[cut:b, 2:]
        want = clean[cut:b, 2:].clone()
        want[..., [5, 40]] = bad
        assert torch.equal(late.isnan(), want.isnan())
        assert torch.equal(late[~late.isnan()], want[~want.isnan()])


def test_no_state_at_all_is_zeros():
    p = Paged([0, 5, 0, 300], 2, 64, 16, "fp16")
    qs = [0, 2, 3, 6, 7]
    q = p.q(7, 4)
    out, err = run(pa.cross, p, q, qs, p.ctx, 0.125)
    assert err == 0
    assert (out[0:2] == 0).all() and (out[3:6] == 0).all()
    compare(out, p, q, qs, p.ctx, 0.125, False)


def test_bad_contexts_give_zeros_and_a_flag():
    p = Paged([100, 100, 100, 100], 1, 64, 16, "bf16")
    q = p.q(20, 2)
    qs = [0, 5, 10, 15, 20]
    cap = p.width * 16
    for call, ctx in ((pa.decode_drafts, [100, 4, 100, 100]), (pa.decode_drafts, [100, 0, 100, 100]),
                      (pa.decode_drafts, [100, -3, 100, 100]), (pa.cross, [100, -1, 100, 100]),
                      (pa.cross, [100, cap + 1, 100, 100]), (pa.decode_drafts, [100, 2 ** 31 - 1, 100, 100])):
        out, err = run(call, p, q, qs, ctx, 0.125)
        assert err == pa.DEVERR_BAD_CONTEXT
        assert (out[5:10] == 0).all()
        for s in (0, 2, 3):
            a, b = qs[s], qs[s + 1]
            ref, mass = attend64(q[a:b], p.k[s], p.v[s], 0.125, 95 if call is pa.decode_drafts else None)
            assert ((out[a:b].double() - ref).abs() <= attention_tolerance(ref, mass, p.dt, 64)).all()


@pytest.mark.parametrize("qs", [[0, 5, 3, 8], [-1, 5, 6, 8], [0, 5, 6, 9], [0, 5, 2 ** 31 - 1, 8]])
def test_impossible_spans_are_left_alone(qs):
    p = Paged([100, 100, 100], 1, 64, 16, "bf16")
    q = p.q(8, 2)
    for call in (pa.decode_drafts, pa.cross):
        out = torch.full_like(q, 7.0).cuda()
        out, err = run(call, p, q, qs, [100] * 3, 0.125, out=out)
        assert err == pa.DEVERR_BAD_CONTEXT
        told = torch.zeros(8, dtype=torch.bool)
        for s in range(3):
            if 0 <= qs[s] <= qs[s + 1] <= 8:
                told[qs[s]:qs[s + 1]] = True
        assert (out[~told] == 7.0).all()


@pytest.mark.parametrize("ctx", [[90, 90], [3000, 90]])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_blocks_give_zeros_and_a_flag(ctx, bad):
    p = Paged(ctx, 2, 128, 16, "bf16")
    caches = p.caches()
    q = p.q(7, 8)
    good = int(p.tables[0, 3])
    p.tables[0, 3] = bad
    for call in (pa.decode_drafts, pa.cross):
        out, err = run(call, p, q, [0, 4, 7], ctx, 0.09, caches=caches)
        assert err == pa.DEVERR_BAD_BLOCK
        assert (out[:4] == 0).all()
        ref, mass = attend64(q[4:], p.k[1], p.v[1], 0.09, ctx[1] - 3 if call is pa.decode_drafts else None)
        assert ((out[4:].double() - ref).abs() <= attention_tolerance(ref, mass, p.dt, 128)).all()
    p.tables[0, 3] = good


def test_blocks_places_change_no_bit():
    ctx, rows = [2500, 77, 640], [5, 3, 40]
    qs = starts(rows)
    outs = []
    for seed in (1, 2):
        p = Paged(ctx, 2, 64, 8, "bf16", seed=9)
        order = torch.randperm(p.nb, generator=torch.Generator().manual_seed(seed))
        p.tables = torch.where(p.tables >= 0, order[p.tables.clamp(min=0).long()].int(), -1)
        q = p.q(qs[-1], 6)
        outs.append([run(c, p, q, qs, ctx, 0.125)[0] for c in (pa.decode_drafts, pa.cross)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_offsets_past_32_bits():
    """Blocks at the far end of a cache of 2^31 and more values."""
    nb = 2 ** 31 // (8 * 16 * 128) + 4096
    kc, vc = (torch.empty(nb, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx, rows = [400, 1000], [3, 2]
    p = Paged(ctx, 8, 128, 16, "bf16", seed=4)
    small = p.caches()
    far = nb - p.nb
    for big, c in zip((kc, vc), small):
        big[far:] = c
    p.tables = torch.where(p.tables >= 0, p.tables + far, -1).int()
    qs = starts(rows)
    q = p.q(qs[-1], 8)
    for causal in (True, False):
        out, err = run(pa.decode_drafts if causal else pa.cross, p, q, qs, ctx, 0.09, caches=(kc, vc))
        assert err == 0
        compare(out, p, q, qs, ctx, 0.09, causal)


def test_padded_batch_and_many_sequences():
    """Hundreds of sequences without rows around a few with some."""
    ctx = [50] * 700
    rows = [0] * 700
    for s, r in ((3, 2), (400, 7), (401, 1), (650, 3)):
        rows[s] = r
    p = Paged(ctx, 1, 64, 16, "fp16", seed=2)
    qs = starts(rows)
    q = p.q(qs[-1] + 5, 2)
    out, err = run(pa.decode_drafts, p, q, qs, ctx, 0.125)
    assert err == 0
    compare(out, p, q, qs, ctx, 0.125, True)


def test_single_tokens_agree_with_decode():
    ctx = [130, 2000, 7, 64]
    p = Paged(ctx, 2, 128, 16, "bf16", seed=12)
    kc, vc = p.caches()
    q = p.q(4, 8)
    a, _ = run(pa.decode_drafts, p, q, [0, 1, 2, 3, 4], ctx, 0.09, caches=(kc, vc))
    b, _ = run(pa.cross, p, q, [0, 1, 2, 3, 4], ctx, 0.09, caches=(kc, vc))
    c = pa.decode(q.cuda(), kc, vc, p.tables.cuda(), i32(ctx), 0.09).cpu()
    assert torch.equal(a, b)
    for s, n in enumerate(ctx):
        ref, mass = attend64(q[s:s + 1], p.k[s], p.v[s], 0.09)
        tol = 2 * attention_tolerance(ref, mass, p.dt, 128)
        assert ((a[s:s + 1].double() - c[s:s + 1].double()).abs() <= tol).all()


def test_captured_and_replayed_with_other_lengths():
    p = Paged([3000, 900, 300], 2, 64, 16, "bf16", seed=15)
    kc, vc = p.caches()
    q = p.q(12, 4)
    dq, tables = q.cuda(), p.tables.cuda()
    ctx, qs = i32([3000, 900, 300]), i32([0, 4, 8, 12])
    work = pa.make_split_workspace(4, 2, 64)
    outs = [torch.empty_like(dq) for _ in range(2)]
    graphs = []
    for call, out in zip((pa.decode_drafts, pa.cross), outs):
        call(dq, kc, vc, tables, ctx, qs, 0.125, out=out, workspace=work)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(dq, kc, vc, tables, ctx, qs, 0.125, out=out, workspace=work)
        graphs.append(g)
    for c, r in (([3000, 900, 300], [4, 4, 4]), ([40, 64, 300], [1, 0, 3]), ([2999, 1, 65], [7, 1, 4])):
        ctx.copy_(i32(c))
        qs.copy_(i32(starts(r)))
        for g in graphs + graphs:  # two graphs, one workspace, one after the other
            g.replay()
        torch.cuda.synchronize()
        p2 = Paged.__new__(Paged)
        p2.__dict__.update(p.__dict__)
        p2.k, p2.v = [k[:n] for k, n in zip(p.k, c)], [v[:n] for v, n in zip(p.v, c)]
        for out, causal in zip(outs, (True, False)):
            compare(out.cpu(), p2, q, starts(r), c, 0.125, causal)
    assert pa.get_device_error() == 0


def test_two_streams_at_once():
    a, b = Paged([4000, 200], 2, 64, 16, "fp16", seed=21), Paged([700, 2500], 2, 64, 16, "fp16", seed=22)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    qs = [0, 5, 9]
    ready = []
    for p in (a, b):
        q = p.q(9, 4)
        ready.append((p, q, q.cuda(), *p.caches(), p.tables.cuda(), i32(p.ctx), i32(qs)))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for (p, q, dq, kc, vc, t, c, s), st in zip(ready, streams):
            with torch.cuda.stream(st):
                outs.append((p, q, pa.decode_drafts(dq, kc, vc, t, c, s, 0.125)))
            outs.append((p, q, pa.decode_drafts(dq, kc, vc, t, c, s, 0.125, stream=st)))
    torch.cuda.synchronize()
    for p, q, out in outs:
        compare(out.cpu(), p, q, qs, p.ctx, 0.125, True)


def test_planned_launch():
    p = Paged([300, 20], 1, 64, 16, "bf16", seed=1)
    kc, vc = p.caches()
    q = p.q(6, 2)
    dq = q.cuda()
    plan = pa.decode_drafts(dq, kc, vc, p.tables.cuda(), i32(p.ctx), i32([0, 2, 6]), 0.125, plan=True)
    for _ in range(2):
        out = plan.run(torch.cuda.current_stream())
        compare(out.cpu(), p, q, [0, 2, 6], p.ctx, 0.125, True)


def test_empty_calls():
    p = Paged([10], 1, 64, 16, "bf16")
    kc, vc = p.caches()
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call in (pa.decode_drafts, pa.cross):
        assert call(none, kc, vc, p.tables.cuda(), i32([10]), i32([0, 0]), 0.1).shape == (0, 2, 64)
        assert call(none, kc, vc, p.tables[:0].cuda(), i32([]), i32([0]), 0.1).shape == (0, 2, 64)


def test_refusals():
    p = Paged([10], 1, 64, 16, "bf16")
    kc, vc = p.caches()
    q = p.q(2, 2).cuda()
    t, c, s = p.tables.cuda(), i32([10]), i32([0, 2])
    for call in (pa.decode_drafts, pa.cross):
        for scale in (0.0, -1.0, math.nan, math.inf):
            with pytest.raises(pa.PagedAttentionError):
                call(q, kc, vc, t, c, s, scale)
        with pytest.raises(pa.PagedAttentionError) as e:
            call(q, kc, vc, t, c, s, 0.1, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
        assert e.value.status == pa.PA_ERR_WORKSPACE
        with pytest.raises(ValueError):
            call(q.half(), kc, vc, t, c, s, 0.1)
        with pytest.raises(ValueError):
            call(q, kc, vc, t, c, i32([0, 1, 2]), 0.1)
        with pytest.raises(ValueError):
            call(q, kc, vc, t, c.cpu(), s, 0.1)
        with pytest.raises(ValueError):
            call(q.transpose(0, 1), kc, vc, t, c, s, 0.1)
        with pytest.raises(ValueError):
            call(q, kc, vc, t, c, s, 0.1, out=torch.empty(2, 2, 64, device="cuda"))
        with pytest.raises(pa.PagedAttentionError):  # 129 query heads to a kv head
            call(p.q(2, 129).cuda(), kc, vc, t, c, s, 0.1,
                 workspace=torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("block", [8, 16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_contexts_up_to_the_tables_end(block, d):
    """A full table, whose last entry is used, of lengths around every tile and block border."""
    for c in (block, 63, 64, 65, 127, 128, 129, 191, 193, 320):
        c = -(-c // block) * block
        p = Paged([c, 1], 2, d, block, "bf16", seed=c)
        p.tables = p.tables[:, :-1].contiguous()
        p.width -= 1
        q = p.q(3, 4)
        for causal in (True, False):
            out, err = run(pa.decode_drafts if causal else pa.cross, p, q, [0, 2, 3], p.ctx, 0.1)
            assert err == 0
            compare(out, p, q, [0, 2, 3], p.ctx, 0.1, causal)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    g = torch.Generator().manual_seed(1000 + seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (), generator=g))
    n = pick(1, 40)
    dtype, d, block = ("bf16", "fp16")[pick(0, 1)], (64, 128)[pick(0, 1)], (8, 16, 32)[pick(0, 2)]
    hkv, G = pick(1, 4), (1, 2, 3, 4, 7, 8, 16)[pick(0, 6)]
    top = (70, 600, 2500)[pick(0, 2)]
    ctx = [pick(1, top) for _ in range(n)]
    rows = [min(c, (pick(0, 4), pick(0, 40), pick(0, 200))[pick(0, 2)]) for c in ctx]
    p = Paged(ctx, hkv, d, block, dtype, seed=seed)
    qs = starts(rows)
    if qs[-1] == 0:
        return
    q = p.q(qs[-1], G * hkv)
    for causal in (True, False):
        out, err = run(pa.decode_drafts if causal else pa.cross, p, q, qs, ctx, 1 / math.sqrt(d))
        assert err == 0
        compare(out, p, q, qs, ctx, 1 / math.sqrt(d), causal)


def test_infinite_scores_and_values_that_are_attended_to():
    """As the formula has it: a score of -inf is no weight, of +inf no number; an infinite value is infinite."""
    p = Paged([300], 1, 64, 16, "bf16", seed=3)
    p.k[0].fill_(1.0)
    q = torch.ones(2, 1, 64, dtype=torch.bfloat16)
    p.k[0][7] = -math.inf
    out, _ = run(pa.cross, p, q, [0, 2], p.ctx, 0.125)
    k = torch.cat([p.v[0][:7], p.v[0][8:]]).double().mean(0)
    assert ((out.double() - k).abs() <= 3 * 2.0 ** -8 * p.v[0].double().abs().mean(0) + 2.0 ** -8 * k.abs()).all()
    p.k[0].fill_(-math.inf)  # no key counts at all: 0 / 0
    out, _ = run(pa.cross, p, q, [0, 2], p.ctx, 0.125)
    assert out.isnan().all()
    p.k[0].fill_(1.0)
    p.k[0][200] = math.inf
    out, _ = run(pa.cross, p, q, [0, 2], p.ctx, 0.125)
    assert out.isnan().all()
    p.k[0].fill_(1.0)
    p.v[0][5, 0, 9] = math.inf
    out, _ = run(pa.cross, p, q, [0, 2], p.ctx, 0.125)
    assert (out[..., 9] == math.inf).all() and out[..., :9].isfinite().all() and out[..., 10:].isfinite().all()


@pytest.mark.parametrize("ctx,rows", [([1500], [1500]), ([3000, 70], [2500, 70]), ([700] * 4, [700, 699, 1, 350])])
def test_prompts_from_scratch(ctx, rows):
    """Pieces of keys that come after every row of their query tile: nothing to add."""
    for dtype, hq, hkv, d in (("bf16", 4, 1, 128), ("fp16", 2, 2, 64)):
        p = Paged(ctx, hkv, d, 16, dtype, seed=13)
        qs = starts(rows)
        q = p.q(qs[-1], hq)
        out, err = run(pa.decode_drafts, p, q, qs, ctx, 0.1)
        assert err == 0
        compare(out, p, q, qs, ctx, 0.1, True)


def test_rows_that_belong_to_no_sequence():
    p = Paged([300, 40], 1, 64, 16, "bf16", seed=4)
    q = p.q(9, 2)
    for call in (pa.decode_drafts, pa.cross):
        out = torch.full_like(q, 7.0).cuda()
        out, err = run(call, p, q, [0, 0, 0], p.ctx, 0.125, out=out)  # nobody has rows
        assert err == 0 and (out == 7.0).all()
        out = torch.full_like(q, 7.0).cuda()
        out, err = run(call, p, q, [2, 5, 6], p.ctx, 0.125, out=out)  # the first two and the last three
        assert err == 0 and (out[[0, 1, 6, 7, 8]] == 7.0).all()
        for s, (a, b) in enumerate(((2, 5), (5, 6))):
            first = p.ctx[s] - (b - a) if call is pa.decode_drafts else None
            ref, mass = attend64(q[a:b], p.k[s], p.v[s], 0.125, first)
            assert ((out[a:b].double() - ref).abs() <= attention_tolerance(ref, mass, p.dt, 64)).all()
