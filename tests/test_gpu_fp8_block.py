"""FP8 blocks with a scale per (block, kv head) on the GPU: the cache write is bit-exact against
the oracle in every form a batch takes; decode is within the bound of its arithmetic of the
float64 oracle over the same codes, and so is prefill; block moves are exact; and the calls run together as a
serving loop makes them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from fp8_block_harness import (DTYPE, Batch, bound, codes_of, dev, dev16, rows16, same_codes, values)
from gpu_harness import device_error
from oracle import fp8_block as fb
from oracle.formats import decode_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def upload(caches):
    return [dev(x) for x in caches]


def same(gpu, want):
    for g, w in zip(gpu[:2], want[:2]):
        same_codes(g, w)
    for g, w in zip(gpu[2:], want[2:4]):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


def append(gpu, key, value, tables, ctx, qs, dtype, **kw):
    return pa.append_fp8_block(dev16(key, dtype), dev16(value, dtype), *gpu, dev(tables),
                               dev(ctx, np.int32), dev(qs, np.int32), **kw)


# ------------------------------------------------------------------------------ cache write

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (8, 128), (5, 64)])
def test_append_in_uneven_parts(dtype, B, hkv, d):
    """Prompts, chunks and single tokens, written in three calls whose parts begin and end
    inside blocks; keys and values grow, so blocks are requantised."""
    b = Batch([1, 7, B, B + 1, 3 * B - 1, 65], hkv, hkv, d, B, dtype, seed=B + d, spread=5)
    caches = b.empty()
    gpu = upload(caches)
    done = np.zeros(len(b.ctx), np.int64)
    for part in range(3):
        left = b.ctx - done
        q = left if part == 2 else b.rng.integers(0, left + 1)
        rows = np.concatenate([np.arange(b.qs[s] + done[s], b.qs[s] + done[s] + q[s]) for s in range(len(q))])
        done = done + q
        qs = np.concatenate([[0], np.cumsum(q)])
        pad = np.concatenate([rows, np.zeros(4, rows.dtype)]).astype(np.int64)  # rows past the last one
        key, value = b.key[pad], b.value[pad]
        caches = fb.append(*caches[:4], key, value, b.tables, done, qs, dtype)
        assert not caches[4]
        append(gpu, key, value, b.tables, done, qs, dtype)
        assert device_error() == 0
        same(gpu, caches)


def test_append_of_many_sequences():
    """More sequences than the scan has threads, with and without new tokens."""
    rng = np.random.default_rng(9)
    n, B = 600, 16
    ctx = rng.integers(1, 40, n)
    b = Batch(ctx, 2, 2, 64, B, "bf16", seed=9, spread=3)
    q = np.minimum(ctx, rng.integers(0, 25, n))
    before = fb.append(*b.empty(), b.key, b.value, b.tables, ctx - q,
                       np.concatenate([[0], np.cumsum(ctx - q)]), "bf16")
    rows = rng.integers(0, len(b.key), q.sum())
    want = fb.append(*before[:4], b.key[rows], b.value[rows], b.tables, ctx, np.concatenate([[0], np.cumsum(q)]), "bf16")
    gpu = upload(before[:4])
    append(gpu, b.key[rows], b.value[rows], b.tables, ctx, np.concatenate([[0], np.cumsum(q)]), "bf16")
    assert device_error() == 0
    same(gpu, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_of_extreme_values(dtype):
    """Zeros, the type's largest and smallest values, infinities and NaN; then a second token
    that raises the scale as far as it goes."""
    top = {"fp16": 0x7BFF, "bf16": 0x7F7F}[dtype]
    inf = {"fp16": 0x7C00, "bf16": 0x7F80}[dtype]
    rows = np.zeros((6, 1, 64), np.uint16)
    rows[1] = 1                      # the smallest subnormal
    rows[2] = top | 0x8000
    rows[3, 0, ::2] = inf
    rows[3, 0, 1] = inf | 0x8001     # NaN
    rows[4, 0, 5] = 0x3C00
    rows[5] = np.arange(64) * 517 % inf
    tables = np.arange(6, dtype=np.int32)[:, None]
    shape = (6, 1, 8, 64)
    caches = (np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8),
              np.zeros(shape[:2], np.float32), np.zeros(shape[:2], np.float32))
    gpu = upload(caches)
    for t in (1, 2):
        more = rows if t == 1 else rows[::-1]
        caches = fb.append(*caches[:4], more, rows, tables, [t] * 6, np.arange(7), dtype)
        append(gpu, more, rows, tables, [t] * 6, np.arange(7), dtype)
        same(gpu, caches)
    assert device_error() == 0


def test_append_refuses_on_the_device():
    """Impossible spans and block ids outside the pool: those writes alone are left out."""
    B, dtype = 16, "fp16"
    b = Batch([20, 20, 20, 20], 2, 2, 64, B, dtype, seed=3, T=3)
    for ctx, qs, tables, bit in [
        ([20, 19, 20, 20], [0, 20, 40, 60, 80], b.tables, pa.DEVERR_BAD_CONTEXT),      # q > c
        ([20, 20, 49, 20], [0, 20, 40, 60, 80], b.tables, pa.DEVERR_BAD_CONTEXT),      # c > T * B
        ([20, 20, 20, 20], [0, 20, 40, 30, 81], b.tables, pa.DEVERR_BAD_CONTEXT),      # decreasing, beyond
        ([20, 20, 20, 20], [-1, 19, 40, 60, 80], b.tables, pa.DEVERR_BAD_CONTEXT),
        ([20, 20, 20, 20], [0, 20, 40, 60, 80],
         np.where(np.arange(3)[None] == 1, [[-1], [3], [b.nb], [4]], b.tables).astype(np.int32), pa.DEVERR_BAD_BLOCK),
    ]:
        tables = tables.copy()
        if bit == pa.DEVERR_BAD_BLOCK:
            tables[1], tables[3] = b.tables[1], b.tables[3]
        caches = b.empty()
        gpu = upload(caches)
        want = fb.append(*caches, b.key, b.value, tables, ctx, qs, dtype)
        append(gpu, b.key, b.value, tables, ctx, qs, dtype)
        assert device_error() == bit and want[4]
        same(gpu, want)


# ------------------------------------------------------------------------------ decode

def check_decode(b, caches, q_bits=None, scale=None, gpu=None):
    scale = 1.0 / np.sqrt(b.d) if scale is None else scale
    q_bits = rows16(b.rng, (len(b.ctx), b.hq, b.d), b.dtype) if q_bits is None else q_bits
    out = pa.decode_fp8_block(dev16(q_bits, b.dtype), *(gpu or upload(caches)), dev(b.tables), dev(b.ctx), scale)
    assert device_error() == 0
    got, q = values(out, b.dtype), decode_bits(q_bits, b.dtype)
    want, errs = fb.paged_decode(q, *caches, b.tables, b.ctx, scale)
    assert not errs.any()
    for s, c in enumerate(b.ctx):
        k = fb.logical_rows(caches[0], caches[2], b.tables[s], c)
        v = fb.logical_rows(caches[1], caches[3], b.tables[s], c)
        off, most = np.abs(got[s] - want[s]), bound(q[s], k, v, scale, want[s], b.dtype)
        assert (off <= most).all(), (s, c, float((off / most).max()))
    return out


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (4, 1, 64), (32, 8, 128), (7, 1, 128), (12, 3, 64),
                                      (10, 5, 128), (32, 2, 64), (40, 2, 128)])
def test_decode_shapes(dtype, B, hq, hkv, d):
    b = Batch([1, 2, B - 1, B, B + 1, 31, 32, 33, 100], hq, hkv, d, B, dtype, seed=hq + B)
    check_decode(b, b.written())


@pytest.mark.parametrize("hq,hkv", [(8, 2), (8, 8), (16, 1)])
@pytest.mark.parametrize("ctx", [[3000], [2000, 1, 700, 1300], [1] * 200])
def test_decode_cut_and_many(hq, hkv, ctx):
    """One sequence cut over every SM, uneven ones, and more sequences than SMs."""
    b = Batch(ctx, hq, hkv, 128, 16, "bf16", seed=len(ctx), spread=2)
    check_decode(b, b.written())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_decode_over_scales_far_apart(dtype, hkv, B):
    """Blocks whose scales differ by 2^8 and more, growing and falling along the context: the
    largest V scale met changes on the way, in pieces and warps of its own."""
    b = Batch([500, 40], 4 * hkv, hkv, 64, B, dtype, seed=B)
    caches = [x.copy() for x in b.written()]
    for s, c in enumerate(b.ctx):
        for j in range(-(-c // B)):
            caches[3][b.tables[s, j]] *= np.exp2((j * 5) % 12 - 6)
            caches[2][b.tables[s, j]] *= np.exp2(-((j * 3) % 4))
    check_decode(b, caches)


def test_decode_over_scales_that_are_no_powers_of_two():
    b = Batch([90, 17], 8, 2, 128, 16, "fp16", seed=2)
    caches = [x.copy() for x in b.written()]
    for c in caches[2:]:
        c *= b.rng.uniform(0.5, 1.9, c.shape).astype(np.float32)
    check_decode(b, caches)


def test_decode_of_invalid_sequences_gives_zeros():
    b = Batch([20, 30, 40, 50], 4, 2, 64, 16, "bf16", seed=5, T=4)
    caches = b.written()
    ctx, tables = b.ctx.copy(), b.tables.copy()
    ctx[0], ctx[1] = 0, 65
    tables[2, 1] = b.nb
    q = rows16(b.rng, (4, 4, 64), "bf16")
    out = values(pa.decode_fp8_block(dev16(q, "bf16"), *upload(caches), dev(tables), dev(ctx), 0.125), "bf16")
    assert device_error() == pa.DEVERR_BAD_CONTEXT | pa.DEVERR_BAD_BLOCK
    assert (out[:3] == 0).all()
    want, _ = fb.paged_decode(decode_bits(q, "bf16"), *caches, b.tables, b.ctx, 0.125)
    assert np.abs(out[3] - want[3]).max() < 0.05


def test_decode_is_the_same_wherever_blocks_sit():
    outs = []
    for seed in (1, 2):
        b = Batch([700, 33, 5], 8, 4, 64, 16, "fp16", seed=1, spread=2)
        perm = np.random.default_rng(seed).permutation(b.nb)
        caches = [np.empty_like(x) for x in b.empty()]
        for c, w in zip(caches, b.written()):
            c[perm] = w
        b.tables = np.where(b.tables >= 0, perm[b.tables], -1).astype(np.int32)
        q = rows16(np.random.default_rng(8), (3, 8, 64), "fp16")
        outs.append(pa.decode_fp8_block(dev16(q, "fp16"), *upload(caches), dev(b.tables), dev(b.ctx), 0.125))
    assert torch.equal(outs[0], outs[1]) and device_error() == 0


def test_decode_graph_stream_and_workspace():
    """A captured decode replayed over changed contexts, on another stream, with a workspace
    of its own, equals plain calls."""
    b = Batch([900, 64, 300], 8, 2, 128, 16, "bf16", seed=11)
    caches = upload(b.written())
    q, tables, ctx = dev16(rows16(b.rng, (3, 8, 128), "bf16"), "bf16"), dev(b.tables), dev(b.ctx)
    ws = pa.make_workspace(8, 2, 128)
    out = torch.empty_like(q)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    plan = pa.decode_fp8_block(q, *caches, tables, ctx, 0.1, out=out, workspace=ws, plan=True)
    plan.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            pa.decode_fp8_block(q, *caches, tables, ctx, 0.1, out=out, workspace=ws, stream=side)
    for lens in ([900, 64, 300], [17, 1, 299], [450, 33, 16]):
        ctx.copy_(dev(lens, np.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, pa.decode_fp8_block(q, *caches, tables, ctx, 0.1))
    assert device_error() == 0


# ------------------------------------------------------------------------------ prefill

def check_prefill(b, new, caches, most=None, scale=None, pad=0):
    """The newest new[s] tokens of every sequence as queries, with `pad` rows behind them."""
    scale = 1.0 / np.sqrt(b.d) if scale is None else scale
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q_bits = rows16(b.rng, (int(qs[-1]) + pad, b.hq, b.d), b.dtype)
    out = torch.full((len(q_bits), b.hq, b.d), 7.0, dtype=DTYPE[b.dtype], device="cuda")
    pa.prefill_fp8_block(dev16(q_bits, b.dtype), *upload(caches), dev(b.tables), dev(b.ctx), dev(qs),
                         scale, int(max(new)) if most is None else most, out=out)
    assert device_error() == 0
    got, q = values(out, b.dtype), decode_bits(q_bits, b.dtype)
    assert (got[int(qs[-1]):] == 7).all()  # rows behind the last sequence stay
    want = fb.paged_prefill(q, *caches, b.tables, b.ctx, qs, scale)
    step = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[b.dtype]  # the weights' own rounding before P V
    for s, c in enumerate(b.ctx):
        k = fb.logical_rows(caches[0], caches[2], b.tables[s], c)
        v = fb.logical_rows(caches[1], caches[3], b.tables[s], c)
        for i in sorted({0, 1, new[s] // 2, new[s] - 2, new[s] - 1} & set(range(new[s]))):
            n = c - (new[s] - 1 - i)
            row = qs[s] + i
            off = np.abs(got[row] - want[row])
            most_off = bound(q[row], k[:n], v[:n], scale, want[row], b.dtype, step)
            assert (off <= most_off).all(), (s, c, i, float((off / most_off).max()))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (8, 2, 64), (7, 1, 128), (12, 4, 128), (16, 1, 64)])
def test_prefill_shapes(dtype, B, hq, hkv, d):
    """Prompts from scratch and chunks, lengths around the tiles and blocks."""
    ctx = [1, B, 63, 64, 65, 129, 200, 333]
    new = [1, B, 5, 64, 65, 129, 77, 1]
    b = Batch(ctx, hq, hkv, d, B, dtype, seed=hq * B, spread=2)
    check_prefill(b, new, b.written(), pad=3)


def test_prefill_long_context_short_query():
    b = Batch([2500, 1030], 8, 2, 128, 16, "bf16", seed=3)
    check_prefill(b, [3, 200], b.written())


def test_prefill_with_empty_and_invalid_sequences():
    b = Batch([40, 70, 90, 30], 4, 2, 64, 16, "fp16", seed=5, T=6)
    caches = b.written()
    new = [0, 70, 20, 30]
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ctx, tables = b.ctx.copy(), b.tables.copy()
    ctx[1] = 69          # more new tokens than context
    tables[2, 0] = -1    # a block outside the pool
    q_bits = rows16(b.rng, (int(qs[-1]), 4, 64), "fp16")
    out = pa.prefill_fp8_block(dev16(q_bits, "fp16"), *upload(caches), dev(tables), dev(ctx), dev(qs), 0.125, 70)
    assert device_error() == pa.DEVERR_BAD_CONTEXT | pa.DEVERR_BAD_BLOCK
    got = values(out, "fp16")
    assert (got[:90] == 0).all()
    want = fb.paged_prefill(decode_bits(q_bits, "fp16"), *caches, b.tables, b.ctx, qs, 0.125)
    assert np.abs(got[90:] - want[90:]).max() < 0.02
    none = pa.prefill_fp8_block(dev16(q_bits, "fp16")[:0], *upload(caches), dev(tables), dev(ctx),
                                dev(np.zeros(5, np.int32)), 0.125, 0)
    assert none.shape == (0, 4, 64) and device_error() == 0


def test_prefill_largest_f16_values():
    """f16 values at the type's end: a code that rounds up past 65504 is clamped, not infinite."""
    b = Batch([20], 2, 1, 64, 16, "fp16", seed=6)
    b.value[:] = 0x7BFF
    caches = b.written()
    assert fb.logical_rows(caches[1], caches[3], b.tables[0], 20).max() == 65536.0
    q = rows16(b.rng, (20, 2, 64), "fp16")
    out = pa.prefill_fp8_block(dev16(q, "fp16"), *upload(caches), dev(b.tables), dev(b.ctx),
                               dev(np.array([0, 20], np.int32)), 0.125, 20)
    got = values(out, "fp16")
    # weights rounded to f16 (2^-11) sum to 1 within 2^-11 and fp32 sums: 65504 (1 +- 2^-10), rounded
    assert device_error() == 0 and np.abs(got - 65504).max() <= 65504 * 2.0 ** -9 and np.isfinite(got).all()
    for ctx in (20, 2000):  # and decode's, whole and cut between SMs
        b = Batch([ctx], 2, 1, 64, 16, "fp16", seed=6)
        b.value[:] = 0x7BFF
        got = values(pa.decode_fp8_block(dev16(q[:1], "fp16"), *upload(b.written()), dev(b.tables), dev(b.ctx), 0.125), "fp16")
        assert device_error() == 0 and np.abs(got - 65504).max() <= 65504 * 2.0 ** -9 and np.isfinite(got).all()


# ------------------------------------------------------------------------------ block moves

@pytest.mark.parametrize("hkv,d,B", [(1, 64, 8), (3, 128, 16), (8, 128, 32), (300, 64, 8)])
def test_copy_blocks(hkv, d, B):
    rng = np.random.default_rng(hkv)
    shape = (9, hkv, B, d)
    caches = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
    caches += [rng.random(shape[:2], dtype=np.float32) for _ in range(2)]
    gpu = upload(caches)
    pairs = np.array([[0, 5], [3, 1], [0, 8], [9, 2], [2, -1]], np.int32)  # the last two are bad
    pa.copy_blocks_fp8_block(*gpu, dev(pairs))
    assert device_error() == pa.DEVERR_BAD_PAIR
    for g, w in zip(gpu, caches):
        w = w.copy()
        w[[5, 1, 8]] = w[[0, 3, 0]]
        np.testing.assert_array_equal(g.cpu().numpy(), w)


def test_swap_out_and_in():
    rng = np.random.default_rng(4)
    shape = (12, 5, 16, 64)
    device = upload([rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
                    + [rng.random(shape[:2], dtype=np.float32) for _ in range(2)])
    saved = [t.clone() for t in device]
    host = [torch.zeros((7, *t.shape[1:]), dtype=t.dtype).pin_memory() for t in device]
    out = torch.tensor([[3, 0], [11, 6], [0, 2]], dtype=torch.int32)
    pa.swap_blocks_fp8_block(device, host, out.cuda())
    torch.cuda.synchronize()
    for t, h in zip(saved, host):
        assert torch.equal(h[[0, 6, 2]], t[[3, 11, 0]].cpu()) and not h[[1, 3, 4, 5]].any()
    for t in device:
        t.zero_()
    pa.swap_blocks_fp8_block(host, device, out.flip(1).contiguous().pin_memory())
    torch.cuda.synchronize()
    for t, was in zip(device, saved):
        assert torch.equal(t[[3, 11, 0]], was[[3, 11, 0]]) and t.float().abs().sum(tuple(range(1, t.dim()))).count_nonzero() == 3
    assert device_error() == 0


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,B,hkv,d", [("bf16", 16, 2, 128), ("fp16", 8, 3, 64)])
def test_a_serving_loop(dtype, B, hkv, d):
    """Prompts, then chunks mixed with single tokens, then decode steps with copy-on-write of a
    forked sequence: tables and slots, write, attention and block copies, with nothing read back
    between the calls of a step; every output against the oracle."""
    rng = np.random.default_rng(B)
    hq, T, nb, scale = 2 * hkv, 24, 96, 1.0 / np.sqrt(d)
    steps = [[30, 0, 17], [40, 21, 1], [1, 5, 1], [1, 1, 1], [1, 1, 1]]
    order = rng.permutation(nb).astype(np.int32)
    tables, free, cells = np.full((3, T), -1, np.int32), dev(order), [dev([0], np.int32), dev([0], np.int32)]
    gt = dev(tables)
    shape = (nb, hkv, B, d)
    caches = (np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8),
              np.full(shape[:2], np.nan, np.float32), np.full(shape[:2], np.nan, np.float32))
    gpu, ctx, start = upload(caches), np.zeros(3, np.int64), 0
    slots = torch.empty(80, dtype=torch.int64, device="cuda")
    for i, new in enumerate(steps):
        ctx = ctx + new
        rows = sum(new) + 2  # a padded batch
        key, value, q = (rows16(rng, (rows, h, d), dtype, 2 if h == hkv else 0) for h in (hkv, hkv, hq))
        if i == 3:  # the last block of sequence 0 was shared with a fork: a copy takes its place
            j = (ctx[0] - 2) // B
            pair = np.array([[tables[0, j], order[-1]]], np.int32)
            pa.copy_blocks_fp8_block(*gpu, dev(pair))
            gt[0, j] = int(order[-1])
            caches = tuple(x.copy() for x in caches[:4])
            for c in caches:
                c[pair[0, 1]] = c[pair[0, 0]]
            tables[0, j] = order[-1]
        lens, news = dev(ctx, np.int32), dev(new, np.int32)
        qs, _ = pa.build_step(news, lens, free, cells[i % 2], gt, B, nb, slots, free_next=cells[1 - i % 2])
        pa.append_fp8_block(dev16(key, dtype), dev16(value, dtype), *gpu, gt, lens, qs)
        out = pa.prefill_fp8_block(dev16(q, dtype), *gpu, gt, lens, qs, scale, max(new))
        one = pa.decode_fp8_block(dev16(q[:3], dtype), *gpu, gt, lens, scale) if max(new) == 1 else None
        tables, ws, wq, start, errs = fb.build_step(new, ctx, order, start, tables, B, nb, 80)
        caches = fb.append(*caches[:4], key, value, tables, ctx, wq, dtype)
        assert not errs and not caches[4]
        assert device_error() == 0
        np.testing.assert_array_equal(gt.cpu().numpy(), tables)
        np.testing.assert_array_equal(slots.cpu().numpy(), ws)
        same(gpu, caches)
        want = fb.paged_prefill(decode_bits(q, dtype), *caches[:4], tables, ctx, wq, scale)
        # values reach 2^2 * 4: within the bound of one output, taken at its largest
        step = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
        for got, row in [(out, None), (one, range(3))]:
            if got is None:
                continue
            got = values(got, dtype)
            for s in range(3):
                k = fb.logical_rows(caches[0], caches[2], tables[s], int(ctx[s]))
                v = fb.logical_rows(caches[1], caches[3], tables[s], int(ctx[s]))
                for r in range(int(wq[s]), int(wq[s + 1])):
                    n = int(ctx[s]) - (int(wq[s + 1]) - 1 - r)
                    most = bound(decode_bits(q[r], dtype), k[:n], v[:n], scale, want[r], dtype, step)
                    assert (np.abs(got[r] - want[r]) <= most).all(), (i, s, r)
