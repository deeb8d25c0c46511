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
