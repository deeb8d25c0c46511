"""verify_drafts against exact arithmetic (whole numbers in the probabilities' own units)."""
from fractions import Fraction
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import i32, starts

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
UNIT = 2 ** 149  # every fp32 value is a whole number of these


def whole(x):
    return [int(Fraction(v) * UNIT) if v > 0 else 0 for v in x.double().tolist()]


def verdict(tokens, target, draft, u):
    """One sequence: (emitted tokens, accepted) by the definition, in exact arithmetic."""
    q, V = len(tokens), target.shape[1]
    a = q - 1
    for i in range(q - 1):
        x = tokens[i + 1]
        d = Fraction(float(draft[i, x])) if draft is not None and 0 <= x < V else 1
        if not (0 <= x < V) or not Fraction(float(u[i])) * d < Fraction(float(target[i, x])):
            a = i
            break
    p = whole(target[a])
    w = list(p)
    if a < q - 1:
        if draft is not None:
            w = [max(x - y, 0) for x, y in zip(p, whole(draft[a]))]
        elif 0 <= tokens[a + 1] < V:
            w[tokens[a + 1]] = 0
        if not any(w):
            w = p
    at = Fraction(float(u[q - 1])) * sum(w)
    run = 0
    for t, x in enumerate(w):
        run += x
        if run > at:
            return tokens[1:a + 1] + [t], a
    return tokens[1:a + 1], a


def make(rows, V, dtype, drawn, seed, sharp=2.0, pad=0, extra=3):
    g = torch.Generator().manual_seed(seed)
    N = sum(rows) + extra
    dt = DTYPES[dtype]
    z = sharp * torch.randn(N, V, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + torch.randn(N, V, generator=g), -1)
    tokens = torch.randint(0, V, (N,), generator=g)
    for r in range(N - 1):  # drawn from the row before, mostly
        if torch.rand((), generator=g) < 0.9:
            tokens[r + 1] = torch.multinomial(q[r], 1, generator=g)[0]
    u = torch.rand(N, generator=g)
    p, q = p.to(dt), q.to(dt)
    if pad:
        p, q = (torch.nn.functional.pad(t, (0, pad), value=math.nan)[:, :V] for t in (p, q))
    return tokens.int(), p, q if drawn else None, u


def check(rows, tokens, p, q, u, ctx=None, **kw):
    qs = starts(rows)
    ctx = ctx or [100 + 3 * s + r for s, r in enumerate(rows)]

    def up(t):
        if t is None:
            return None
        big = torch.empty(t.shape[0], t.stride(0), dtype=t.dtype)
        big[:, :t.shape[1]] = t
        big = big.cuda()
        return big[:, :t.shape[1]]
    out = torch.full_like(tokens, -7).cuda()
    pa.get_device_error()
    out, emitted, left = pa.verify_drafts(tokens.cuda(), up(p), up(q), u.cuda(), i32(qs), i32(ctx), out=out, **kw)
    assert pa.get_device_error() == 0
    out, emitted, left = out.tolist(), emitted.tolist(), left.tolist()
    for s, r in enumerate(rows):
        a, b = qs[s], qs[s + 1]
        if r == 0:
            assert emitted[s] == 0 and left[s] == ctx[s]
            continue
        want, _ = verdict(tokens[a:b].tolist(), p[a:b], None if q is None else q[a:b], u[a:b])
        assert out[a:b] == want + [-1] * (r - len(want)), s
        assert emitted[s] == len(want) and left[s] == ctx[s] - r + len(want)
    assert all(x == -7 for x in out[qs[-1]:])


@pytest.mark.parametrize("V", [1, 2, 127, 128, 129, 1000, 4096, 5003])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("drawn", [True, False])
def test_against_exact_arithmetic(V, dtype, drawn):
    rows = [1, 4, 2, 0, 8, 3, 1, 5]
    check(rows, *make(rows, V, dtype, drawn, seed=V + drawn))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_padded_rows(dtype):
    """Rows farther apart than the vocabulary, NaN between; aligned and not."""
    for pad in (1, 24):
        rows = [3, 1, 6]
        check(rows, *make(rows, 1000, dtype, True, seed=5, pad=pad))


def test_a_large_vocabulary():
    rows = [2, 1, 4]
    check(rows, *make(rows, 128256, "fp32", True, seed=1))


def test_many_drafts():
    rows = [300, 1, 700]
    tokens, p, q, u = make(rows, 50, "fp32", True, seed=3)
    check(rows, tokens, p, q, u)
    check(rows, tokens, p, p.clone(), u)  # the same model: all accepted


def test_borders():
    """Sums that hit the drawn number exactly, numbers at the ends, weights of zero around them."""
    V = 600
    p = torch.zeros(4, V)
    p[:, 200], p[:, 201], p[:, 400] = 0.25, 0.25, 0.5
    rows = [1, 1, 1, 1]
    tokens = torch.zeros(4, dtype=torch.int32)
    for u, want in ((0.0, 200), (0.25, 201), (0.24999999, 200), (0.5, 400), (0.49999997, 201), (1 - 2.0 ** -24, 400)):
        out = pa.verify_drafts(tokens.cuda(), p.cuda(), None, torch.full((4,), u, device="cuda"), i32([0, 1, 2, 3, 4]),
                               i32([1] * 4))[0]
        assert out.tolist() == [want] * 4
    for u in (1.0, 2.0):  # past the last sum: the last token with a weight
        out = pa.verify_drafts(tokens.cuda(), p.cuda(), None, torch.full((4,), u, device="cuda"), i32([0, 1, 2, 3, 4]),
                               i32([1] * 4))[0]
        assert out.tolist() == [400] * 4
    for u in (-0.5, math.nan):  # as 0
        out = pa.verify_drafts(tokens.cuda(), p.cuda(), None, torch.full((4,), u, device="cuda"), i32([0, 1, 2, 3, 4]),
                               i32([1] * 4))[0]
        assert out.tolist() == [200] * 4
    # u d == p is a refusal, a hair less is not
    p2 = torch.tensor([[0.5, 0.5, 0.0], [0.0, 0.0, 1.0]]).cuda()
    d2 = torch.tensor([[0.0, 1.0, 0.0], [0.0, 0.0, 0.0]]).cuda()
    for u, want in ((0.5, [0, -1]), (0.5 - 2.0 ** -25, [1, 2])):
        out = pa.verify_drafts(i32([0, 1]), p2, d2, torch.tensor([u, 0.3], device="cuda"), i32([0, 2]), i32([9]))[0]
        assert out.tolist() == want


def test_nothing_left_over_draws_from_the_target():
    p = torch.tensor([[0.25, 0.25, 0.5], [0.1, 0.2, 0.7]]).cuda()
    d = torch.tensor([[0.25, 0.25, 1.0], [0.0, 0.0, 1.0]]).cuda()
    out, emitted, left = pa.verify_drafts(i32([5, 2]), p, d, torch.tensor([0.9, 0.3], device="cuda"), i32([0, 2]), i32([7]))
    assert out.tolist() == [1, -1] and emitted.tolist() == [1] and left.tolist() == [6]
    # a certain draft with all of the target's weight cannot be refused; one without any is
    p = torch.tensor([[0.0, 1.0], [1.0, 0.0]]).cuda()
    for x, want in ((1, [1, 0]), (0, [1, -1])):
        out = pa.verify_drafts(i32([0, x]), p, None, torch.tensor([0.99, 0.5], device="cuda"), i32([0, 2]), i32([7]))[0]
        assert out.tolist() == want


def test_odd_probabilities():
    """What is negative or no number counts as 0, above 1 as 1; rows of large sums do not overflow."""
    V = 300
    p = torch.full((1, V), math.nan)
    p[0, 10], p[0, 20], p[0, 30], p[0, 40] = -1.0, math.inf, 1.0, -math.inf
    for u, want in ((0.0, 20), (0.49, 20), (0.5, 30), (0.99, 30)):
        out = pa.verify_drafts(i32([0]), p.cuda(), None, torch.tensor([u], device="cuda"), i32([0, 1]), i32([1]))[0]
        assert out.tolist() == [want]
    ones = torch.ones(1, 100000).cuda()
    for u in (0.0, 0.25, 0.5, 0.75, 0.999):
        out = pa.verify_drafts(i32([0]), ones, None, torch.tensor([u], device="cuda"), i32([0, 1]), i32([1]))[0]
        assert out.tolist() == [int(float(torch.tensor(u)) * 100000)]


def test_no_probability_at_all_is_told():
    p = torch.zeros(3, 500).cuda()
    p[0, 7] = 1.0
    pa.get_device_error()
    out, emitted, left = pa.verify_drafts(i32([1, 7, 3]), p, None, torch.full((3,), 0.5, device="cuda"), i32([0, 3]), i32([20]))
    assert pa.get_device_error() == pa.DEVERR_BAD_PROBS
    assert out.tolist() == [7, -1, -1] and emitted.tolist() == [1] and left.tolist() == [18]


def test_tokens_outside_the_vocabulary_are_refused():
    rows = [3, 2]
    tokens, p, q, u = make(rows, 100, "fp32", True, seed=2)
    for bad in (-1, 100, 2 ** 31 - 1):
        tokens[1] = tokens[4] = bad
        check(rows, tokens, p, q, u)
        check(rows, tokens, p, None, u)


def test_impossible_sequences():
    tokens, p, q, u = make([2, 2, 2], 100, "fp32", True, seed=2, extra=0)
    for qs, ctx in (([0, 2, 4, 7], [9, 9, 9]), ([0, 2, 4, 6], [9, 9, 1]), ([-1, 2, 4, 6], [9, 9, 9])):
        out = torch.full_like(tokens, -7).cuda()
        pa.get_device_error()
        out, emitted, left = pa.verify_drafts(tokens.cuda(), p.cuda(), q.cuda(), u.cuda(), i32(qs), i32(ctx), out=out)
        assert pa.get_device_error() == pa.DEVERR_BAD_CONTEXT
        bad = 0 if qs[0] < 0 else 2
        assert emitted[bad] == 0 and left[bad] == ctx[bad]
        assert (out[4:] == -7).all() if bad == 2 else (out[:2] == -7).all()
        assert emitted[1] > 0


def test_lengths_in_place_plan_and_graph():
    rows = [4, 1, 3]
    tokens, p, q, u = make(rows, 1000, "fp32", True, seed=11, extra=0)
    qs, ctx = i32(starts(rows)), i32([50, 60, 70])
    want = pa.verify_drafts(tokens.cuda(), p.cuda(), q.cuda(), u.cuda(), qs, ctx)
    live = ctx.clone()
    emitted = torch.zeros(3, dtype=torch.int32, device="cuda")
    plan = pa.verify_drafts(tokens.cuda(), p.cuda(), q.cuda(), u.cuda(), qs, live, emitted=emitted, context_next=live,
                            plan=True)
    out = plan.run(torch.cuda.current_stream())
    assert torch.equal(out, want[0]) and torch.equal(emitted, want[1]) and torch.equal(live, want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(torch.cuda.current_stream())
    live.copy_(ctx)
    out.zero_()
    g.replay()
    assert torch.equal(out, want[0]) and torch.equal(live, want[2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pa.verify_drafts(tokens.cuda(), p.cuda(), q.cuda(), u.cuda(), qs, ctx, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    tokens, p, q, u = (t.cuda() for t in make([3], 100, "fp32", True, seed=2, extra=0))
    qs, ctx = i32([0, 3]), i32([9])
    with pytest.raises(ValueError):
        pa.verify_drafts(tokens.long(), p, q, u, qs, ctx)
    with pytest.raises(ValueError):
        pa.verify_drafts(tokens, p, q[:, :50], u, qs, ctx)
    with pytest.raises(ValueError):
        pa.verify_drafts(tokens, p, q.half(), u, qs, ctx)
    with pytest.raises(ValueError):
        pa.verify_drafts(tokens, p.t().contiguous().t(), q, u, qs, ctx)
    with pytest.raises(ValueError):
        pa.verify_drafts(tokens, p[:2], q[:2], u, qs, ctx)
    with pytest.raises(TypeError):
        pa.verify_drafts(tokens, p.double(), q.double(), u, qs, ctx)
    with pytest.raises(pa.PagedAttentionError):  # the output over the input
        pa.verify_drafts(tokens, p, q, u, qs, ctx, out=tokens)
    with pytest.raises(pa.PagedAttentionError):
        pa.verify_drafts(tokens, torch.empty(3, 2 ** 20 + 1, device="cuda"), None, u, qs, ctx)
    empty = pa.verify_drafts(tokens[:0], p[:0], None, u[:0], i32([0, 0, 0]), i32([4, 5]))
    assert empty[1].tolist() == [0, 0] and empty[2].tolist() == [4, 5]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("pads,offsets", [((1, 2), (0, 0)), ((3, 3), (1, 3)), ((7, 16), (5, 0)), ((8, 8), (0, 1))])
def test_rows_that_start_anywhere(dtype, pads, offsets):
    """Target and draft rows at their own distances and places within 16 bytes."""
    rows, V = [3, 1, 6, 2], 1003
    tokens, p, q, u = make(rows, V, dtype, True, seed=17)
    views = []
    for t, pad, off in zip((p, q), pads, offsets):
        flat = torch.full((t.shape[0] * (V + pad) + off,), math.nan, dtype=t.dtype)
        view = flat[off:].view(t.shape[0], V + pad)[:, :V]
        view.copy_(t)
        views.append(flat.cuda()[off:].view(t.shape[0], V + pad)[:, :V])
    qs = starts(rows)
    for d in (views[1], None):
        pa.get_device_error()
        out, emitted, _ = pa.verify_drafts(tokens.cuda(), views[0], d, u.cuda(), i32(qs), i32([50] * 4))
        assert pa.get_device_error() == 0
        for s, r in enumerate(rows):
            a, b = qs[s], qs[s + 1]
            want, _ = verdict(tokens[a:b].tolist(), p[a:b], None if d is None else q[a:b], u[a:b])
            assert out[a:b].tolist() == want + [-1] * (r - len(want)) and emitted[s] == len(want)


def test_the_largest_vocabulary():
    V = 2 ** 20
    p = torch.zeros(2, V)
    p[:, [0, 511, 512, 600000, V - 1]] = torch.tensor([0.125, 0.125, 0.25, 0.25, 0.25])
    for u, want in ((0.0, 0), (0.125, 511), (0.25, 512), (0.5, 600000), (0.75, V - 1), (0.99, V - 1)):
        out = pa.verify_drafts(i32([1, 2]), p.cuda(), None, torch.full((2,), u, device="cuda"), i32([0, 1, 2]), i32([1, 1]))[0]
        assert out.tolist() == [want] * 2


@pytest.mark.parametrize("n", [1, 77, 160, 400, 700])
def test_batches_of_every_cluster_size(n):
    """8, 4, 2 and 1 CTAs to a sequence give the same tokens."""
    rows = [2] * n
    tokens, p, q, u = make([2, 2, 2, 2], 900, "fp32", True, seed=23, extra=0)
    rep = -(-n // 4)
    check(rows, tokens.repeat(rep)[:2 * n], p.repeat(rep, 1)[:2 * n], q.repeat(rep, 1)[:2 * n], u.repeat(rep)[:2 * n])


def test_two_streams_at_once():
    rows = [3, 1, 4]
    batches = [make(rows, 5000, "fp32", True, seed=s, extra=0) for s in (31, 32)]
    qs, ctx = i32(starts(rows)), i32([20, 20, 20])
    up = [[t.cuda() for t in b] for b in batches]
    want = [pa.verify_drafts(*b, qs, ctx)[0].clone() for b in up]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        for i in (0, 1):
            got.append((i, pa.verify_drafts(*up[i], qs, ctx, stream=streams[i])[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i, t in got)
