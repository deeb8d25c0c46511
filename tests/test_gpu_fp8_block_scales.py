"""FP8 blocks whose scales lie far apart: what a token does not attend to, or attends to with no
weight to speak of, does not move its output, however large that block's scale is.

The bound here is the arithmetic's own, whatever the output's type: weights are rounded to f16
once, and what f16 cannot hold of them is measured by the largest weighted scale that the query
meets, not by the largest scale."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from fp8_block_harness import HALF_STEP, Batch, dev, dev16, rows16, values
from gpu_harness import device_error
from oracle import fp8_block as fb
from oracle.formats import decode_bits, encode_bits

pytestmark = pytest.mark.gpu

SMALLEST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the type's subnormals
LARGEST = {"fp16": 65504.0, "bf16": 2.0 ** 128 - 2.0 ** 120}


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def upload(caches):
    return [dev(x) for x in caches]


def rows_of(b, caches, s, n):
    """K, V and V's scales [n, Hkv, ...] of sequence s's first n tokens."""
    k = fb.logical_rows(caches[0], caches[2], b.tables[s], n)
    v = fb.logical_rows(caches[1], caches[3], b.tables[s], n)
    sv = caches[3][b.tables[s, np.arange(n) // b.B]].astype(np.float64)
    return k, v, sv


def expected(q, k, v, sv, scale, dtype, odd=False):
    """(output, how far a kernel may be from it) of one query.  q [Hq, d], k, v [n, Hkv, d], sv
    [n, Hkv] float64.  With weights w (softmax), per output element:
      * the output's own rounding, half a step;
      * weights rounded once to f16 before P V, 2^-11 of sum w |v|;
      * a weight off by delta_t because its score is: d exact products summed in fp32 (tensor cores
        add with at least 2^-22 relative to the terms' magnitudes each; bf16 rows of q, brought to
        f16's upper range, those of a kv head together in decode, lose 2^-39 of their largest
        value at most), two fp32 factors, an exp2 off by 2^-22 and its argument's rounding:
        numerator and denominator;
      * n sums in fp32 and rescalings, n 2^-22;
      * the base-2 logarithm of V's scale joins the exponent and leaves it again, two roundings in
        fp32 of up to twice its size: 2^-22 of it;
      * weights times their block's scale that f16 holds as subnormals: 2^-25 each against the
        largest weighted scale rounded up to a power of two, W, times the code;
      * odd: scales that are no powers of two go through a base-2 logarithm of two units in
        the last place, 2^-16."""
    n, hkv, d = k.shape
    out, most = np.empty(q.shape), np.empty(q.shape)
    for h in range(q.shape[0]):
        g = h // (q.shape[0] // hkv)
        kh, vh, sh = k[:, g], v[:, g], sv[:, g]
        z = scale * (kh @ q[h])
        w = np.exp(z - z.max())
        w /= w.sum()
        out[h] = w @ vh
        delta = (abs(scale) * (d * 2.0 ** -22 * (np.abs(kh) @ np.abs(q[h]))
                               + 2.0 ** -39 * np.abs(q.reshape(hkv, -1)[g]).max() * np.abs(kh).sum(1))
                 + 2.0 ** -21 * np.abs(z) + 2.0 ** -22 * (z.max() - z) + 2.0 ** -21)
        rel = 2.0 ** -11 + (n + np.abs(np.log2(sh)).max()) * 2.0 ** -22 + (2.0 ** -16 if odd else 0)
        code = np.abs(vh) / sh[:, None]
        most[h] = ((rel * (w @ np.abs(vh)) + (w * delta) @ (np.abs(vh) + np.abs(out[h]))
                    + 2.0 ** -24 * (w * sh).max() * code.sum(0)) * (1 + HALF_STEP[dtype])
                   + HALF_STEP[dtype] * np.abs(out[h]) + SMALLEST[dtype])
    return np.clip(out, -LARGEST[dtype], LARGEST[dtype]), most


def check(b, caches, got, q, qs, scale, rows=None, odd=False):
    """got [rows, Hq, d] float64 of the queries q, sequence s's at rows qs[s] .. qs[s + 1] - 1 (its
    newest tokens), against each row's own sum over the cache."""
    for s, c in enumerate(int(x) for x in b.ctx):
        new = int(qs[s + 1] - qs[s])
        for i in range(new) if rows is None else sorted(set(rows) & set(range(new))):
            k, v, sv = rows_of(b, caches, s, c - (new - 1 - i))
            want, most = expected(q[qs[s] + i], k, v, sv, scale, b.dtype, odd)
            off = np.abs(got[qs[s] + i] - want)
            assert (off <= most).all(), (s, c, i, float((off / most).max()))


def prefill(b, caches, q_bits, new, scale):
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = pa.prefill_fp8_block(dev16(q_bits, b.dtype), *upload(caches), dev(b.tables), dev(b.ctx),
                               dev(qs), scale, int(max(new)))
    assert device_error() == 0
    return values(out, b.dtype), decode_bits(q_bits, b.dtype), qs


# ------------------------------------------------------------------------------ prefill

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,hq,hkv,d", [(8, 4, 2, 128), (16, 8, 2, 128), (16, 4, 1, 64), (32, 3, 3, 64)])
@pytest.mark.parametrize("grow", [12, 30, 110])
def test_a_later_block_of_any_scale_does_not_move_earlier_tokens(dtype, B, hq, hkv, d, grow):
    """Blocks further on in the same key tile whose K or V scale is larger by 2^grow: the tokens
    before them give the same bits, and every token what its own keys give."""
    b = Batch([200, 70], hq, hkv, d, B, dtype, seed=B + grow)
    plain = b.written()
    q_bits = rows16(b.rng, (270, hq, d), dtype)
    scale = 1.0 / np.sqrt(d)
    want, q, qs = prefill(b, plain, q_bits, [200, 70], scale)
    check(b, plain, want, q, qs, scale, rows=(0, 40, 69, 199))
    at = 32  # a block boundary for every B, inside the first key tile
    for which in (2, 3):
        caches = [x.copy() for x in plain]
        for s in range(2):
            caches[which][b.tables[s, at // B]] *= np.float32(2.0 ** grow)
            if s == 0:
                caches[which][b.tables[s, 128 // B]] *= np.float32(2.0 ** min(2 * grow, 115))
        got, _, _ = prefill(b, caches, q_bits, [200, 70], scale)
        for s in range(2):
            early = slice(int(qs[s]), int(qs[s]) + at)
            np.testing.assert_array_equal(got[early], want[early])
        if which == 3 and dtype == "bf16":  # (a K scale as large gives scores past fp32's use)
            check(b, caches, got, q, qs, scale, rows=(0, 31, 32, 33, 63, 64, 127, 128, 199))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,d", [(8, 64), (16, 128), (32, 128)])
def test_prefill_over_scales_at_random(dtype, B, d):
    """V scales over 2^-40 .. 2^40 and K scales over 2^8, block by block, in no order."""
    b = Batch([500, 130], 4, 2, d, B, dtype, seed=d + B)
    caches = [x.copy() for x in b.written()]
    low, high = (-40, 41) if dtype == "bf16" else (-6, 7)
    for s in range(2):
        for blk in b.tables[s, :-(-int(b.ctx[s]) // B)]:
            caches[3][blk] *= np.exp2(b.rng.integers(low, high, 2)).astype(np.float32)
            caches[2][blk] *= np.exp2(b.rng.integers(-8, 1, 2)).astype(np.float32)
    q_bits = rows16(b.rng, (430, 4, d), dtype)
    got, q, qs = prefill(b, caches, q_bits, [300, 130], 1.0 / np.sqrt(d))
    check(b, caches, got, q, qs, 1.0 / np.sqrt(d), rows=(0, 1, 17, 63, 64, 100, 129, 211, 299))


def unseen(b, s, j, q_row, far):
    """K rows of block j of sequence s that every head scores `far` below the others: against the
    query that all heads share."""
    k = -far * q_row / (q_row @ q_row)
    return np.broadcast_to(k, (b.B, b.hkv, b.d))


def negligible(dtype, B, hq, hkv, d, ctx, far, seed):
    """A batch whose heads share a query, the codes of one block (number 2) against it, and
    everything else ordinary; the score's unit is `scale` = 1."""
    b = Batch([ctx, 120], hq, hkv, d, B, dtype, seed=seed)
    q_row = b.rng.choice([-1.0, 1.0], d) * 0.25
    for s in range(2):
        at = slice(int(b.qs[s]) + 2 * B, int(b.qs[s]) + 3 * B)
        b.key[at] = encode_bits(unseen(b, s, 2, q_row, far), dtype)
    return b, q_row, [x.copy() for x in b.written()]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,hq,hkv,d", [(8, 4, 2, 64), (16, 8, 2, 128), (32, 4, 1, 128)])
@pytest.mark.parametrize("far,grow", [(60, 30), (20, 22), (12, 14)])
def test_prefill_of_a_large_block_without_weight(dtype, B, hq, hkv, d, far, grow):
    """A block whose V scale is larger by 2^grow and whose weight is e^-far of the others'."""
    b, q_row, caches = negligible(dtype, B, hq, hkv, d, 400, far, far)
    for s in range(2):
        caches[3][b.tables[s, 2]] *= np.float32(2.0 ** grow)
    q_bits = encode_bits(np.broadcast_to(q_row, (520, hq, d)).copy(), dtype)
    got, q, qs = prefill(b, caches, q_bits, [400, 120], 1.0)
    check(b, caches, got, q, qs, 1.0, rows=(3 * B, 3 * B + 1, 119, 150, 399))


@pytest.mark.parametrize("low,high", [(-100, 120), (-140, -126), (-130, 90), (100, 120)])
def test_prefill_over_the_whole_range_of_scales(low, high):
    """bf16 outputs over V scales that alternate between the ends of the range that the write
    stores, and past it (subnormal floats, in a cache made elsewhere)."""
    b = Batch([150], 4, 2, 128, 16, "bf16", seed=7)
    caches = [x.copy() for x in b.written()]
    np.copyto(caches[1], caches[1] & 0xBF, where=(caches[1] & 0x7F) != 0x7F)  # (codes below 2)
    for j in range(10):
        caches[3][b.tables[0, j]] = np.float32(2.0 ** (low if (j // 2) % 2 == 0 else high))
    q_bits = rows16(b.rng, (150, 4, 128), "bf16")
    got, q, qs = prefill(b, caches, q_bits, [150], 0.09)
    assert np.isfinite(got).all()
    check(b, caches, got, q, qs, 0.09, rows=(0, 15, 31, 32, 40, 64, 100, 149))


# ------------------------------------------------------------------------------ decode

def decode(b, caches, q_bits, scale):
    out = pa.decode_fp8_block(dev16(q_bits, b.dtype), *upload(caches), dev(b.tables), dev(b.ctx), scale)
    assert device_error() == 0
    return values(out, b.dtype), decode_bits(q_bits, b.dtype), np.arange(len(b.ctx) + 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,hq,hkv,d", [(8, 8, 8, 64), (16, 8, 2, 128), (32, 16, 1, 128), (16, 32, 8, 128)])
@pytest.mark.parametrize("ctx", [150, 3000])
@pytest.mark.parametrize("far,grow", [(60, 30), (20, 22), (12, 14)])
def test_decode_of_a_large_block_without_weight(dtype, B, hq, hkv, d, ctx, far, grow):
    """A block whose V scale is larger by 2^grow and whose weight is e^-far of the others', in
    sequences of one piece and of many."""
    b, q_row, caches = negligible(dtype, B, hq, hkv, d, ctx, far, far)
    for s in range(2):
        caches[3][b.tables[s, 2]] *= np.float32(2.0 ** grow)
    q_bits = encode_bits(np.broadcast_to(q_row, (2, hq, d)).copy(), dtype)
    got, q, qs = decode(b, caches, q_bits, 1.0)
    check(b, caches, got, q, qs, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,hq,hkv,d", [(8, 8, 8, 64), (16, 8, 2, 128), (32, 16, 1, 128), (16, 7, 1, 64)])
@pytest.mark.parametrize("ctx", [[130, 7, 33], [2500]])
def test_decode_over_scales_at_random(dtype, B, hq, hkv, d, ctx):
    """V scales over 2^-40 .. 2^40 and K scales over 2^8, block by block, in no order."""
    b = Batch(ctx, hq, hkv, d, B, dtype, seed=d + B)
    caches = [x.copy() for x in b.written()]
    low, high = (-40, 41) if dtype == "bf16" else (-6, 7)
    for s, c in enumerate(ctx):
        for blk in b.tables[s, :-(-c // B)]:
            caches[3][blk] *= np.exp2(b.rng.integers(low, high, hkv)).astype(np.float32)
            caches[2][blk] *= np.exp2(b.rng.integers(-8, 1, hkv)).astype(np.float32)
    q_bits = rows16(b.rng, (len(ctx), hq, d), dtype)
    got, q, qs = decode(b, caches, q_bits, 1.0 / np.sqrt(d))
    check(b, caches, got, q, qs, 1.0 / np.sqrt(d))


@pytest.mark.parametrize("hq,hkv", [(8, 8), (4, 1), (16, 1)])
@pytest.mark.parametrize("ctx", [100, 2600])
@pytest.mark.parametrize("low,high", [(-100, 120), (-140, -126), (-130, 90), (100, 120)])
def test_decode_over_the_whole_range_of_scales(hq, hkv, ctx, low, high):
    """bf16 outputs over V scales that alternate between the ends of the range that the write
    stores, and past it (subnormal floats, in a cache made elsewhere); the first sequence has the
    lower end alone."""
    b = Batch([30, ctx], hq, hkv, 128, 16, "bf16", seed=7)
    caches = [x.copy() for x in b.written()]
    np.copyto(caches[1], caches[1] & 0xBF, where=(caches[1] & 0x7F) != 0x7F)  # (codes below 2)
    for s in range(2):
        for j in range(-(-int(b.ctx[s]) // 16)):
            caches[3][b.tables[s, j]] = np.float32(2.0 ** (low if (j // 2) % 2 == 0 else high))
    q_bits = rows16(b.rng, (2, hq, 128), "bf16")
    got, q, qs = decode(b, caches, q_bits, 0.09)
    assert np.isfinite(got).all()
    check(b, caches, got, q, qs, 0.09)


@pytest.mark.parametrize("hq,hkv", [(8, 8), (4, 1), (32, 2)])
@pytest.mark.parametrize("ctx", [40, 3000])
def test_decode_of_values_whose_sum_passes_fp32(hq, hkv, ctx):
    """Values near bf16's largest: their sum over the context is no float, their average is."""
    b = Batch([ctx], hq, hkv, 64, 16, "bf16", seed=3)
    b.value[:] = np.where(b.value & 0x8000, 0xFEC0, 0x7EC0)  # +-1.5 * 2^126
    caches = b.written()
    q_bits = rows16(b.rng, (1, hq, 64), "bf16")
    got, q, qs = decode(b, caches, q_bits, 0.125)
    assert np.isfinite(got).all()
    check(b, caches, got, q, qs, 0.125)
    b.value[:] = 0x7F00  # 2^127
    caches = b.written()
    got, q, qs = decode(b, caches, q_bits, 0.125)
    check(b, caches, got, q, qs, 0.125)


def test_decode_of_one_long_sequence_of_the_largest_values():
    """300000 values of 2^127 in every warp of every SM: their average is 2^127."""
    ctx, B, d = 300000, 16, 64
    gen, nb = torch.Generator(device="cuda").manual_seed(1), 300000 // 16
    k8 = torch.randint(0, 0x50, (nb, 1, B, d), generator=gen, device="cuda", dtype=torch.uint8)  # up to 12
    v8 = torch.full_like(k8, 0x70)  # 128
    ks, vs = torch.full((nb, 1), 0.125, device="cuda"), torch.full((nb, 1), 2.0 ** 120, device="cuda")
    q = torch.randn(1, 1, d, generator=gen, device="cuda").bfloat16()
    out = pa.decode_fp8_block(q, k8, v8, ks, vs, torch.arange(nb, dtype=torch.int32, device="cuda")[None],
                              dev([ctx], np.int32), 0.125)
    # weights rounded to f16 (2^-11) over unrounded sums, and 2^-22 for each of the sums
    most = 2.0 ** 127 * (2.0 ** -11 + ctx * 2.0 ** -22 + HALF_STEP["bf16"])
    assert device_error() == 0 and np.abs(values(out, "bf16") - 2.0 ** 127).max() <= most


# ------------------------------------------------------------------------------ queries

@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (4, 1, 64), (32, 2, 128)])
@pytest.mark.parametrize("ctx", [60, 2000])
@pytest.mark.parametrize("up", [-90, -30, -13, 17, 60])
def test_queries_of_any_size(hq, hkv, d, ctx, up):
    """bf16 queries 2^up times as large over keys 2^-up times as large have the same scores, to the
    bit, in decode and in prefill; each row has a power of two of its own, and a row of zeros."""
    b = Batch([ctx, 90], hq, hkv, d, 16, "bf16", seed=11)
    plain = b.written()
    q = decode_bits(rows16(b.rng, (2, hq, d), "bf16", spread=3), "bf16")
    q[1, 0] = 0.0
    scale, outs = 1.0 / np.sqrt(d), []
    for e in (0, up):
        caches = [x.copy() for x in plain]
        caches[2] = np.ldexp(caches[2], -e).astype(np.float32)
        q_bits = encode_bits(np.ldexp(q, e), "bf16")
        got, qf, qs = decode(b, caches, q_bits, scale)
        check(b, caches, got, qf, qs, scale)
        again, _, _ = prefill(b, caches, q_bits, [1, 1], scale)
        check(b, caches, again, qf, qs, scale)
        outs.append((got, again))
    np.testing.assert_array_equal(outs[0][0], outs[1][0])
    np.testing.assert_array_equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (32, 2, 64), (20, 1, 128)])
def test_queries_of_different_sizes_in_a_group(hq, hkv, d):
    """Heads of one kv head whose queries lie up to 2^24 apart."""
    b = Batch([70, 900], hq, hkv, d, 16, "bf16", seed=13)
    caches = b.written()
    q = decode_bits(rows16(b.rng, (2, hq, d), "bf16"), "bf16")
    q = np.ldexp(q, np.linspace(-20, 4, hq).round().astype(int)[None, :, None])
    for order in (slice(None), slice(None, None, -1)):
        q_bits = encode_bits(np.ascontiguousarray(q[:, order]), "bf16")
        got, qf, qs = decode(b, caches, q_bits, 1.0 / np.sqrt(d))
        check(b, caches, got, qf, qs, 1.0 / np.sqrt(d))
        got, qf, qs = prefill(b, caches, q_bits, [1, 1], 1.0 / np.sqrt(d))
        check(b, caches, got, qf, qs, 1.0 / np.sqrt(d))


def test_a_query_that_is_not_finite_reaches_its_head_and_no_other():
    b = Batch([100, 2000], 8, 2, 128, 16, "bf16", seed=12)
    caches = b.written()
    q_bits = rows16(b.rng, (2, 8, 128), "bf16")
    plain = pa.decode_fp8_block(dev16(q_bits, "bf16"), *upload(caches), dev(b.tables), dev(b.ctx), 0.1)
    for what in (0x7F80, 0xFF80, 0x7FC0):
        odd = q_bits.copy()
        odd[:, 5, 77] = what
        out = pa.decode_fp8_block(dev16(odd, "bf16"), *upload(caches), dev(b.tables), dev(b.ctx), 0.1)
        assert torch.isnan(out[:, 5]).all()
        keep = [0, 1, 2, 3, 4, 6, 7]
        assert torch.equal(out[:, keep], plain[:, keep]) and device_error() == 0


# ------------------------------------------------------------------------------ one rounding

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (8, 2, 64), (7, 1, 128), (12, 4, 128), (16, 1, 64), (64, 1, 128)])
def test_weights_are_rounded_once_to_f16_whatever_the_outputs_type(dtype, B, hq, hkv, d):
    """Ordinary batches: prompts from scratch, chunks and single tokens around the tiles and blocks."""
    ctx, new = [1, B, 63, 64, 65, 129, 200, 333], [1, B, 5, 64, 65, 129, 77, 1]
    b = Batch(ctx, hq, hkv, d, B, dtype, seed=hq * B + 1, spread=2)
    caches, scale = b.written(), 1.0 / np.sqrt(d)
    q_bits = rows16(b.rng, (sum(new), hq, d), dtype)
    got, q, qs = prefill(b, caches, q_bits, new, scale)
    check(b, caches, got, q, qs, scale, rows=(0, 1, 32, 76, 128))
    got, q, qs = decode(b, caches, q_bits[:len(ctx)], scale)
    check(b, caches, got, q, qs, scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,hq,hkv,d", [(8, 4, 2, 64), (16, 8, 2, 128), (32, 16, 1, 128)])
def test_scales_that_are_no_powers_of_two(dtype, B, hq, hkv, d):
    """A cache made elsewhere, over a range of 2^12: codes are exact whatever the scale is."""
    b = Batch([300, 77], hq, hkv, d, B, dtype, seed=B)
    caches = [x.copy() for x in b.written()]
    for c in caches[2:]:
        c *= np.exp2(b.rng.uniform(-6, 6, c.shape)).astype(np.float32)
    caches[2] *= np.float32(2.0 ** -4)
    q_bits, scale = rows16(b.rng, (277, hq, d), dtype), 1.0 / np.sqrt(d)
    got, q, qs = prefill(b, caches, q_bits, [200, 77], scale)
    check(b, caches, got, q, qs, scale, rows=(0, 17, 76, 150, 199), odd=True)
    got, q, qs = decode(b, caches, q_bits[:2], scale)
    check(b, caches, got, q, qs, scale, odd=True)


@pytest.mark.parametrize("ctx,at", [(30, 3), (100, 99), (700, 40), (700, 650)])
def test_the_weight_of_a_key_that_stands_out_is_not_rounded(ctx, at):
    """One key scores e^17 and more above the others, by another fraction in each sequence: its
    weight is 1 within 2^-14, so an fp16 output is its value to half a step, whichever tile it is
    in.  (Scales that are no powers of two, so that the values are no fp16 numbers; their base-2
    logarithms are off by 2^-16.)"""
    n, hq, hkv, d, B = 24, 8, 4, 128, 16
    b = Batch([ctx] * n, hq, hkv, d, B, "fp16", seed=ctx + at)
    q_row = b.rng.choice([-1.0, 1.0], d) * 0.25
    b.key[:] = encode_bits(decode_bits(b.key, "fp16") * 2.0 ** -6, "fp16")
    for s in range(n):
        b.key[int(b.qs[s]) + at] = encode_bits(np.broadcast_to((18 + s / 24) * q_row / (q_row @ q_row), (hkv, d)), "fp16")
    caches = [x.copy() for x in b.written()]
    caches[3] *= b.rng.uniform(1, 2, caches[3].shape).astype(np.float32)
    q_bits = encode_bits(np.broadcast_to(q_row, (n, hq, d)).copy(), "fp16")
    got, q, qs = decode(b, caches, q_bits, 1.0)
    again, _, _ = prefill(b, caches, q_bits, [1] * n, 1.0)
    for s in range(n):
        k, v, _ = rows_of(b, caches, s, ctx)
        top = v[at].repeat(hq // hkv, 0)
        z = np.stack([k[:, h // 2] @ q[s, h] for h in range(hq)], 1)
        rest = np.delete(np.exp(z - z.max(0)), at, 0).sum(0)[:, None]
        assert (rest < 2.0 ** -14).all()
        half = np.spacing(np.abs(top).astype(np.float16)).astype(np.float64) / 2
        most = half * (1 + 2.0 ** -10) + 2.0 ** -16 * np.abs(top) + (rest + 2.0 ** -20) * 2 * np.abs(v).max()
        assert (np.abs(got[s] - top) <= most).all() and (np.abs(again[s] - top) <= most).all(), s
