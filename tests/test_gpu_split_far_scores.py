"""decode_drafts and cross where scores are so large that a rounding of their size is many powers of
two: whatever finite scores are, the largest of a row has the weight 1."""
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import DT, Paged, attend64, attention_tolerance, run, starts

pytestmark = pytest.mark.gpu
# q's and k's first values, scale: scores exact in fp32, of some 2^14 to 2^120 in log2 units and past fp32's range
SIZES = [("fp16", 128.0, 128.0, 1.0), ("fp16", 4096.0, 4096.0, 1.0), ("fp16", 6000.0, 6000.0, 128 * 0.088),
         ("fp16", 16384.0, 32768.0, 0.7), ("fp16", 65504.0, -65504.0, 1.0), ("fp16", 65504.0, 65504.0, 100.0),
         ("fp16", 10.0, 3.0, 1e37), ("bf16", 2.0 ** 12, 2.0 ** 13, 0.3), ("bf16", 2.0 ** 20, -2.0 ** 20, 0.125),
         ("bf16", 2.0 ** 60, 2.0 ** 60, 1.0), ("bf16", 1.0, 1.0, 1e37)]
CTX, ROWS = [1, 5, 200, 3000, 700], [1, 3, 9, 5, 150]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 2)])
@pytest.mark.parametrize("wide", [False, True])
def test_equal_scores_of_any_size_weigh_alike(size, d, hkv, wide):
    """Every score of a row is the same number: the mean of the values it attends to."""
    dtype, a, b, scale = size
    ctx, rows = (CTX, ROWS) if wide else (CTX[:4], ROWS[:4])
    p = Paged(ctx, hkv, d, 16, dtype, seed=31)
    qs = starts(rows)
    q = torch.zeros(qs[-1], 4 * hkv, d, dtype=DT[dtype])
    q[..., 0] = a
    for k in p.k:
        k.zero_()
        k[..., 0] = b
    for call in (pa.decode_drafts, pa.cross):
        out, err = run(call, p, q, qs, ctx, scale)
        assert err == 0
        for s, c in enumerate(ctx):
            x, y = qs[s], qs[s + 1]
            ref, mass = attend64(q[x:y], p.k[s], p.v[s], 1.0, c - (y - x) if call is pa.decode_drafts else None)
            assert ((out[x:y].double() - ref).abs() <= attention_tolerance(ref, mass, p.dt, d)).all(), (s, call)


@pytest.mark.parametrize("dtype,a,scale", [("fp16", 65504.0, 1.0), ("fp16", 60000.0, 50.0), ("bf16", 2.0 ** 40, 1.0),
                                           ("fp16", 8.0, 1e37), ("bf16", 2.0 ** 100, 0.1)])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_of_far_scores_takes_the_weight(dtype, a, scale, rising, d):
    """Keys in steps far apart, from small ones on, rising (a new maximum in every tile and piece) or falling: each
    row's output is the value of its largest score."""
    ctx, rows = [700, 60, 2100], [4, 9, 140]
    p = Paged(ctx, 1, d, 16, dtype, seed=32)
    qs = starts(rows)
    q = torch.zeros(qs[-1], 2, d, dtype=DT[dtype])
    q[..., 0] = a
    top = {"fp16": 60000.0, "bf16": 2.0 ** 20}[dtype]
    where = []
    for s, c in enumerate(ctx):
        # a step every 32 keys, each a value of its own in the type, among keys of the smallest score
        step = torch.linspace(1.0, top, -(-c // 32)).to(DT[dtype])
        if not rising:
            step = step.flip(0)
        p.k[s].zero_()
        p.k[s][..., 0] = -top
        p.k[s][::32, 0, 0] = step
        where.append(list(range(0, c, 32)))
    for call in (pa.decode_drafts, pa.cross):
        out, err = run(call, p, q, qs, ctx, scale)
        assert err == 0
        for s, c in enumerate(ctx):
            x, y = qs[s], qs[s + 1]
            for i in range(y - x):
                last = c - (y - x) + i if call is pa.decode_drafts else c - 1
                t = max(k for k in where[s] if k <= last) if rising else 0
                # (one weight of 1: exact)
                assert torch.equal(out[x + i], p.v[s][t].expand(2, d)), (s, i, t)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("base", [2.0 ** 10, 2832.0, 2.0 ** 16, 2.0 ** 19])
def test_small_differences_of_far_scores(dtype, base):
    """Scores base + 0 .. 12, exact in fp32: the weights are those of the differences."""
    ctx, rows = [1000, 3000, 90], [5, 2, 50]
    d = 64
    p = Paged(ctx, 1, d, 16, dtype, seed=33)
    qs = starts(rows)
    q = torch.zeros(qs[-1], 2, d, dtype=DT[dtype])
    q[..., 0], q[..., 1] = 128.0, 1.0
    g = torch.Generator().manual_seed(7)
    small = []
    for s, c in enumerate(ctx):
        p.k[s].zero_()
        p.k[s][..., 1] = torch.randint(0, 13, (c, 1), generator=g).to(DT[dtype])
        small.append(p.k[s].clone())
        p.k[s][..., 0] = base / 128
    for call in (pa.decode_drafts, pa.cross):
        out, err = run(call, p, q, qs, ctx, 1.0)
        assert err == 0
        for s, c in enumerate(ctx):
            x, y = qs[s], qs[s + 1]
            ref, mass = attend64(q[x:y], small[s], p.v[s], 1.0, c - (y - x) if call is pa.decode_drafts else None)
            # below 2^12 (in log2 units) a row's reference is its largest score scaled and rounded, past it the score
            # itself: where a row's largest passes that border (base 2832), and where pieces on both sides of it are joined,
            # weights are off by half a step of a number below 2^13, 2^-12, times ln 2, once each; all the others' sum
            # is off by as much
            extra = 2 * math.log(2) * 2.0 ** -12 if base == 2832.0 else 0.0
            tol = attention_tolerance(ref, mass, p.dt, d) + 2 * extra * mass
            assert ((out[x:y].double() - ref).abs() <= tol).all(), (s, call)


@pytest.mark.parametrize("dtype,a,b", [("fp16", 16384.0, 32768.0), ("bf16", 2.0 ** 30, -2.0 ** 10)])
@pytest.mark.parametrize("ctx,rows", [([40], [9]), ([3000, 90], [9, 3]), ([700, 90], [200, 60])])
@pytest.mark.parametrize("d", [64, 128])
def test_far_rows_beside_keys_not_attended(dtype, a, b, ctx, rows, d):
    """V of a later draft that is not finite changes no bit of the rows before it where scores are far, too."""
    p = Paged(ctx, 1, d, 16, dtype, seed=34)
    qs = starts(rows)
    q = torch.zeros(qs[-1], 2, d, dtype=DT[dtype])
    q[..., 0] = a
    for k in p.k:
        k.zero_()
        k[..., 0] = b
    clean, err = run(pa.decode_drafts, p, q, qs, ctx, 0.5)
    assert err == 0
    odd = [5, d - 3]
    at = [c - r + r // 2 for c, r in zip(ctx, rows)]
    for s, t in enumerate(at):
        p.v[s][t, 0, odd] = math.nan
    out, err = run(pa.decode_drafts, p, q, qs, ctx, 0.5)
    assert err == 0
    for s, t in enumerate(at):
        cut, end = qs[s] + t - (ctx[s] - rows[s]), qs[s + 1]
        assert torch.equal(out[qs[s]:cut], clean[qs[s]:cut])
        want = torch.zeros(d, dtype=torch.bool)
        want[odd] = True
        assert torch.equal(out[cut:end].isnan(), want.expand(end - cut, 2, d))
