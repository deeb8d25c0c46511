"""verify_drafts of what is no probability and no uniform number, and of the smallest probabilities.

A probability that is negative or no number counts as 0, one above 1 as 1, a uniform number below 0
or no number as 0 and, in a draft's test, one above 1 as 1: in the tests of the drafts as in the
sums."""
import itertools
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import i32
from test_gpu_verify import DTYPES, verdict

pytestmark = pytest.mark.gpu
ODD = [0.0, -0.0, 0.25, 0.5, 1.0, 2.0, -1.0, math.nan, math.inf, -math.inf]
UNIFORMS = [0.0, 0.5, 1 - 2.0 ** -24, 1.0, 3.0, math.inf, -0.5, -math.inf, math.nan]


def counted(t):
    return torch.where(t.isnan(), torch.zeros_like(t), t).clamp(0.0, 1.0) + 0.0


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("drawn", [True, False])
def test_drafts_are_tested_by_what_counts(dtype, drawn):
    """Every pair of odd values at the drafted token, with every odd uniform number."""
    dt = DTYPES[dtype]
    cases = list(itertools.product(ODD, ODD if drawn else [1.0], UNIFORMS))
    n = len(cases)
    p, q, u = torch.zeros(2 * n, 3), torch.zeros(2 * n, 3), torch.full((2 * n,), 0.3)
    p[0::2] = torch.tensor([[0.5, pt, 0.25] for pt, _, _ in cases])
    q[0::2] = torch.tensor([[0.25, d, 0.125] for _, d, _ in cases])
    p[1::2, 2] = 1.0
    u[0::2] = torch.tensor([x for _, _, x in cases])
    p, q = p.to(dt), q.to(dt)
    tokens = torch.ones(2 * n, dtype=torch.int32)
    pa.get_device_error()
    out, emitted, left = pa.verify_drafts(tokens.cuda(), p.cuda(), q.cuda() if drawn else None, u.cuda(),
                                          i32(range(0, 2 * n + 1, 2)), i32([9] * n))
    assert pa.get_device_error() == 0
    out, emitted, left = out.tolist(), emitted.tolist(), left.tolist()
    cp, cq, cu = counted(p), counted(q), counted(u)
    for s, case in enumerate(cases):
        a, b = 2 * s, 2 * s + 2
        want, _ = verdict([1, 1], cp[a:b], cq[a:b] if drawn else None, cu[a:b])
        assert out[a:b] == want + [-1] * (2 - len(want)), case
        assert emitted[s] == len(want) and left[s] == 7 + len(want), case


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_smallest_probabilities(dtype):
    """Probabilities count in whole units of 2^-54, rounded to nearest with ties to even: 2^-55 and less is 0,
    for the sampled token, for what a refused draft leaves over and for a row's having any at all."""
    unit, V, dt = 2.0 ** -54, 700, DTYPES[dtype]

    def sample(entries, u):
        p = torch.zeros(1, V)
        for t, x in entries:
            p[0, t] = x
        pa.get_device_error()
        out, emitted, _ = pa.verify_drafts(i32([0]), p.to(dt).cuda(), None, torch.tensor([u], device="cuda"), i32([0, 1]),
                                           i32([5]))
        return out.tolist(), emitted.tolist(), pa.get_device_error()
    none = ([-1], [0], pa.DEVERR_BAD_PROBS)
    for x, there in ((unit, True), (0.75 * unit, True), (0.5 * unit, False), (0.25 * unit, False), (2.0 ** -126, False)):
        assert sample([(7, x)], 0.5) == (([7], [1], 0) if there else none)
        assert sample([(t, x) for t in range(V)], 0.0) == (([0], [1], 0) if there else none)
        assert sample([(7, x), (600, 4 * unit)], 0.0) == ([7 if there else 600], [1], 0)
    # 1.5 units are two: of three, the first two are token 7's
    assert sample([(7, 1.5 * unit), (9, unit)], 0.5)[0] == [7]
    assert sample([(7, 1.5 * unit), (9, unit)], 0.7)[0] == [9]

    def refused(target, draft):  # token 1 is refused; from what it leaves over, or the target where that is nothing
        p, d = torch.zeros(2, V), torch.zeros(2, V)
        for t, x in target:
            p[0, t] = x
        for t, x in draft:
            d[0, t] = x
        pa.get_device_error()
        out = pa.verify_drafts(i32([0, 1]), p.to(dt).cuda(), d.to(dt).cuda(), torch.tensor([0.5, 0.5], device="cuda"),
                               i32([0, 2]), i32([5]))[0]
        assert pa.get_device_error() == 0
        return out.tolist()
    draft = [(0, 0.5), (1, 1.0)]
    assert refused([(0, 0.5), (2, unit)], draft) == [2, -1]
    assert refused([(0, 0.5), (2, 0.75 * unit)], draft) == [2, -1]
    assert refused([(0, 0.5), (2, 0.5 * unit)], draft) == [0, -1]
    # target and draft are rounded one by one: 1.5 units less 0.75 are 2 - 1, 1.25 less 0.75 are 1 - 1
    assert refused([(0, 0.5), (3, 1.5 * unit)], draft + [(3, 0.75 * unit)]) == [3, -1]
    assert refused([(0, 0.5), (3, 1.25 * unit)], draft + [(3, 0.75 * unit)]) == [0, -1]
