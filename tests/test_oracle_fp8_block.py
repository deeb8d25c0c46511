"""The oracle of FP8 blocks with block scales and of a step's bookkeeping, pinned on the CPU:
the scale rule against its definition, values against exact cases and torch's E4M3
conversion, growth against a rewrite, attention against the 16-bit oracle on values that
E4M3 holds, and tables and slots against the block pool."""
import numpy as np
import pytest
import torch

from oracle import attention, fp8, fp8_block as fb
from oracle.block_pool import BlockPool
from oracle.formats import decode_bits, encode_bits


def empty(nb, hkv, B, d):
    return (np.full((nb, hkv, B, d), 0x7F, np.uint8), np.full((nb, hkv, B, d), 0x7F, np.uint8),
            np.zeros((nb, hkv), np.float32), np.zeros((nb, hkv), np.float32))


@pytest.mark.parametrize("amax", [0.0, 2.0 ** -133, 1e-30, 0.875, np.nextafter(0.875, 1), 1.0, 447.0,
                                  448.0, 449.0, 65504.0, 3.38e38])
def test_scale_exponent_is_the_smallest(amax):
    e = fb.scale_exponent(amax)
    assert fb.LOWEST <= e <= fb.HIGHEST
    assert amax <= 448 * 2.0 ** e
    assert e == fb.LOWEST or amax > 448 * 2.0 ** (e - 1)


def test_values_are_torchs_e4m3_of_the_scaled_input():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((20, 2, 64)) * np.exp2(rng.integers(-9, 9, (20, 2, 1)))).astype(np.float16)
    bits = x.view(np.uint16)
    k8, v8, ks, vs = empty(4, 2, 16, 64)
    tables = np.array([[2, 0]], np.int32)
    k8, v8, ks, vs, errs = fb.append(k8, v8, ks, vs, bits, bits, tables, [20], [0, 20], "fp16")
    assert not errs
    for b, rows in ((2, x[:16]), (0, x[16:])):
        for h in range(2):
            s = ks[b, h]
            top = np.abs(rows[:, h].astype(np.float64)).max()
            assert np.log2(s) % 1 == 0 and 224 * s < top <= 448 * s
            want = torch.from_numpy(rows[:, h].astype(np.float32) / s).to(torch.float8_e4m3fn)
            np.testing.assert_array_equal(k8[b, h, :len(rows)], want.view(torch.uint8).numpy())
    assert (k8[0, :, 4:] == 0x7F).all() and (k8[1] == 0x7F).all() and (ks[1] == 0).all()
    np.testing.assert_array_equal(k8, v8)


def test_growth_equals_one_write_but_for_subnormals():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((9, 1, 64)) * np.exp2(np.arange(9))[:, None, None]).astype(np.float16)
    bits, tables = x.view(np.uint16), np.array([[1]], np.int32)
    once = fb.append(*empty(2, 1, 16, 64), bits, bits, tables, [9], [0, 9], "fp16")
    grown = empty(2, 1, 16, 64)
    for t in range(9):
        grown = fb.append(*grown[:4], bits[t:t + 1], bits[t:t + 1], tables, [t + 1], [0, 1], "fp16")
    np.testing.assert_array_equal(once[2], grown[2])
    a, b = fp8.decode_e4m3(once[0][1, 0, :9]), fp8.decode_e4m3(grown[0][1, 0, :9])
    normal = np.abs(a) >= 2.0 ** -5
    np.testing.assert_array_equal(a[normal], b[normal])
    assert np.abs(a - b).max() <= 2.0 ** -9  # a subnormal code moves by one step at most


def test_a_write_from_row_zero_begins_the_block_anew():
    k8, v8, ks, vs = empty(1, 1, 8, 64)
    ks[:], vs[:] = 2.0 ** 60, np.nan
    bits = np.full((1, 1, 64), 0x3C00, np.uint16)  # 1.0
    k8, v8, ks, vs, _ = fb.append(k8, v8, ks, vs, bits, bits, np.zeros((1, 1), np.int32), [1], [0, 1], "fp16")
    assert ks[0, 0] == vs[0, 0] == 2.0 ** -8 and (fp8.decode_e4m3(k8[0, 0, 0]) == 256).all()


def test_values_that_are_not_finite():
    x = np.array([np.nan, np.inf, -np.inf, 1.75] + [0.0] * 60, np.float16)
    bits = x.view(np.uint16).reshape(1, 1, 64)
    k8, _, ks, _, _ = fb.append(*empty(1, 1, 8, 64), bits, bits, np.zeros((1, 1), np.int32), [1], [0, 1], "fp16")
    got = fp8.decode_e4m3(k8[0, 0, 0, :4])
    assert ks[0, 0] == 2.0 ** -8 and np.isnan(got[0]) and list(got[1:]) == [448, -448, 448]


def test_attention_over_exact_values_is_the_16_bit_oracle():
    rng = np.random.default_rng(5)
    rows = rng.integers(-8, 9, (21, 2, 64)) / 8.0  # multiples of 1/8 up to 1: exact in E4M3
    bits = encode_bits(rows, "bf16")
    tables = np.array([[3, 1, 0]], np.int32)
    k8, v8, ks, vs, _ = fb.append(*empty(4, 2, 8, 64), bits, bits, tables, [21], [0, 21], "bf16")
    k16 = np.zeros((4, 2, 8, 64), np.uint16)
    for t in range(21):
        k16[tables[0, t // 8], :, t % 8] = bits[t]
    q = rng.standard_normal((5, 4, 64))
    want = [attention.attend(q[i], rows[:17 + i], rows[:17 + i], 0.125) for i in range(5)]
    got = fb.paged_prefill(q, k8, v8, ks, vs, tables, [21], [0, 5], 0.125)
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-14)
    one, err = fb.paged_decode(q[4:], k8, v8, ks, vs, tables, [21], 0.125)
    np.testing.assert_allclose(one[0], want[4], rtol=0, atol=1e-14)
    np.testing.assert_array_equal(decode_bits(k16[3], "bf16"), fp8.decode_e4m3(k8[3]) * ks[3][:, None, None])
    assert not err.any()


def test_build_step_takes_the_blocks_that_the_pool_takes():
    rng = np.random.default_rng(6)
    B, nb = 16, 64
    order = rng.permutation(nb).astype(np.int32)
    pool = BlockPool(nb, B, order)
    past = [0, 5, 16, 31, 0]
    new = [33, 1, 1, 2, 0]
    tables = np.full((5, 6), -7, np.int32)
    for s, p in enumerate(past):
        if p:
            pool.allocate(s, p)
            tables[s, :-(-p // B)] = pool.block_table(s)
    used = sum(-(-p // B) for p in past)
    got, slots, starts, nxt, errs = fb.build_step(new, np.add(past, new), order, used, tables, B, nb, 40)
    assert not errs and list(starts) == [0, 33, 34, 35, 37, 37] and (slots[37:] == -1).all()
    pool.allocate(0, 33)
    for s in (1, 2, 3):
        for _ in range(new[s]):
            pool.append_slot(s)
    at = 0
    for s in range(4):
        t = pool.block_table(s)
        assert list(got[s, :len(t)]) == list(t) and (got[s, len(t):] == -7).all()
        assert [pool.slot(s, past[s] + i) for i in range(new[s])] == list(slots[at:at + new[s]])
        at += new[s]
    assert nxt == used + 3 + 1 + 1


@pytest.mark.parametrize("why", ["blocks", "slots"])
def test_build_step_is_all_or_nothing(why):
    tables = np.full((2, 2), -1, np.int32)
    free = np.arange(4, dtype=np.int32)
    start, slots = (3, 40) if why == "blocks" else (0, 31)
    got, s, starts, nxt, errs = fb.build_step([16, 16], [16, 16], free, start, tables, 16, 4, slots)
    assert errs == {why} and nxt == start and (s == -1).all() and (got == tables).all()
    assert list(starts) == [0, 16, 32]
