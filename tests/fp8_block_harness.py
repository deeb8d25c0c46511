"""Batches over FP8 blocks with block scales for the GPU tests: random tables, caches written
by the oracle, and the bound that an attention output may be off by."""
import numpy as np
import torch

from oracle import fp8_block as fb
from oracle.fp8 import decode_e4m3
from oracle.formats import decode_bits, encode_bits

DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}  # rounding, relative to the value


def dev(x, dtype=None):
    x = np.ascontiguousarray(x if dtype is None else np.asarray(x, dtype=dtype))
    return torch.from_numpy(x).cuda()


def dev16(bits, dtype):
    return dev(bits.view(np.int16)).view(DTYPE[dtype])


def host16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def rows16(rng, shape, dtype, spread=0):
    """16-bit patterns of normal values, each (token, head) with a power of two of its own."""
    gain = np.exp2(rng.integers(-spread, spread + 1, (*shape[:-1], 1)))
    return encode_bits(rng.standard_normal(shape) * gain, dtype)


class Batch:
    """Sequences of the given contexts in a shuffled pool whose unwritten rows hold NaN codes
    and whose unwritten scales hold NaN."""

    def __init__(self, ctx, hq, hkv, d, B, dtype, seed=0, spread=0, T=None):
        rng = np.random.default_rng(seed)
        self.ctx, self.hq, self.hkv, self.d, self.B, self.dtype = np.array(ctx, np.int32), hq, hkv, d, B, dtype
        used = -(-self.ctx // B)
        self.T = T or int(used.max()) + 1
        self.nb = int(used.sum()) + 3
        order, at = rng.permutation(self.nb).astype(np.int32), 0
        self.tables = np.full((len(ctx), self.T), -1, np.int32)
        for s, u in enumerate(used):
            self.tables[s, :u] = order[at:at + u]
            at += u
        self.qs = np.concatenate([[0], np.cumsum(self.ctx)]).astype(np.int32)
        total = int(self.qs[-1])
        self.key = rows16(rng, (total, hkv, d), dtype, spread)
        self.value = rows16(rng, (total, hkv, d), dtype, spread)
        self.rng = rng

    def empty(self):
        shape = (self.nb, self.hkv, self.B, self.d)
        nan = np.full(shape[:2], np.nan, np.float32)
        return np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8), nan, nan.copy()

    def written(self):
        """Caches with every context written at once, by the oracle."""
        out = fb.append(*self.empty(), self.key, self.value, self.tables, self.ctx, self.qs, self.dtype)
        assert not out[4]
        return out[:4]


def bound(q, k, v, scale, ref, dtype, p_step=2.0 ** -11):
    """How far a kernel's output for one query may be from `ref`, by its arithmetic.  q [Hq, d],
    k, v [ctx, Hkv, d] float64 (dequantised).  With weights w (softmax), per output element:
      * the output's own rounding, half a step of |ref|;
      * weights rounded once before P V: p_step (half a step of that type) of sum w |v|;
      * weights off because scores are: a score is a sum of d exact products in fp32 (tensor
        cores add with at least 2^-22 relative to the terms' magnitudes each), scaled by two
        fp32 factors, its exp2 off by 2^-22: a weight is off by delta = (d * 2^-22 *
        max_t scale sum |q k_t| + 2^-21 max |z|) + 2^-21 relative, numerator and denominator;
      * sums of ctx weights and products in fp32, and the rescalings of the running maximum,
        ctx * 2^-22 relative in all;
      * weights below 2^-14 rounded in f16's subnormals: 2^-25 each, times the largest |v| of
        the scale's range (2 amax), over the sum of the weights, which is at least one."""
    ctx, hkv = k.shape[:2]
    out = np.empty(q.shape)
    for h in range(q.shape[0]):
        kh, vh = k[:, h // (q.shape[0] // hkv)], v[:, h // (q.shape[0] // hkv)]
        z = scale * (kh @ q[h])
        w = np.exp(z - z.max())
        w /= w.sum()
        spread = w @ np.abs(vh)
        delta = (q.shape[1] * 2.0 ** -22 * abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
                 + 2.0 ** -21 * np.abs(z).max() + 2.0 ** -21)
        out[h] = (HALF_STEP[dtype] * np.abs(ref[h])
                  + (p_step + 2 * delta + ctx * 2.0 ** -22) * (1 + HALF_STEP[dtype]) * spread
                  + ctx * 2.0 ** -25 * 2 * np.abs(vh).max())
    return out + 2.0 ** -24  # (f16 outputs below its normals)


def values(t, dtype):
    return decode_bits(host16(t), dtype)


def codes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def same_codes(got, want):
    """Equal codes, NaN of either sign alike."""
    g, w = codes_of(got), want
    nan = (w & 0x7F) == 0x7F
    np.testing.assert_array_equal(np.where(nan, 0, g), np.where(nan, 0, w))
    np.testing.assert_array_equal(np.isnan(decode_e4m3(g)), nan)
