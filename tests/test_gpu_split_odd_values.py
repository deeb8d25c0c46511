"""decode_drafts beside values of V that are not finite, at both head sizes and in both halves of a row."""
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import Paged, run, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [8, 32])
@pytest.mark.parametrize("ctx,rows", [([40], [9]), ([3000], [9]), ([9000, 64], [5, 1]), ([700, 90], [200, 60]),
                                      ([2100] * 3, [150, 140, 300])])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_of_later_rows_change_no_bit(d, block, ctx, rows, bad):
    """One token's V is not finite in some columns: the rows before it keep their bits, those from it on get it, in
    whole items and cut ones, with one query tile and two."""
    dtype, G = ("bf16", 4) if block == 8 else ("fp16", 3)
    p = Paged(ctx, 2, d, block, dtype, seed=41)
    qs = starts(rows)
    q = p.q(qs[-1], 2 * G)
    clean, err = run(pa.decode_drafts, p, q, qs, ctx, 0.125)
    assert err == 0
    odd = [0, 5, 31, 33, d // 2 + 6, d - 1]
    at = [c - r + r // 2 for c, r in zip(ctx, rows)]
    for s, t in enumerate(at):
        p.v[s][t, 1, odd] = bad
    out, err = run(pa.decode_drafts, p, q, qs, ctx, 0.125)
    assert err == 0
    for s, t in enumerate(at):
        a, cut, b = qs[s], qs[s] + t - (ctx[s] - rows[s]), qs[s + 1]
        assert torch.equal(out[a:cut], clean[a:cut])
        want = clean[cut:b].clone()
        want[:, G:, odd] = bad
        assert torch.equal(out[cut:b].isnan(), want.isnan())
        assert torch.equal(out[cut:b].nan_to_num(7.0), want.nan_to_num(7.0))
