"""Calls of the FP8 block-scale step that follow one another with nothing between them: each launch
may begin while the one before it ends, and reads what that one wrote; and calls with nothing to do."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from fp8_block_harness import Batch, dev, dev16, rows16, same_codes
from gpu_harness import device_error
from oracle import fp8_block as fb
from oracle.formats import decode_bits, encode_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def upload(caches):
    return [dev(x) for x in caches]


@pytest.mark.parametrize("dtype,n,hkv,d,B", [("bf16", 200, 2, 64, 16), ("fp16", 90, 8, 128, 8)])
def test_writes_that_follow_one_another(dtype, n, hkv, d, B):
    """40 single tokens to each sequence, growing, so that blocks are requantised again and again:
    40 calls in a row, every code and scale as the oracle's."""
    steps = 40
    rng = np.random.default_rng(n)
    past = rng.integers(0, 30, n)
    b = Batch(past + steps, hkv, hkv, d, B, dtype, seed=n)
    key, value = (rows16(rng, (steps, n, hkv, d), dtype) for _ in range(2))
    grow = np.exp2(np.arange(steps) // 3)[:, None, None, None]
    key, value = (encode_bits(decode_bits(x, dtype) * grow, dtype) for x in (key, value))
    qs = np.arange(n + 1, dtype=np.int32)
    starts = np.concatenate([[0], np.cumsum(past)])
    caches = fb.append(*b.empty(), b.key[:starts[-1]], b.value[:starts[-1]], b.tables, past, starts, dtype)
    gpu = upload(caches[:4])
    args = [(dev16(key[i], dtype), dev16(value[i], dtype), dev(past + i + 1, np.int32)) for i in range(steps)]
    tables, rows = dev(b.tables), dev(qs)
    torch.cuda.synchronize()
    for k, v, lens in args:
        pa.append_fp8_block(k, v, *gpu, tables, lens, rows)
    assert device_error() == 0
    for i in range(steps):
        caches = fb.append(*caches[:4], key[i], value[i], b.tables, past + i + 1, qs, dtype)
    for g, w in zip(gpu[:2], caches[:2]):
        same_codes(g, w)
    for g, w in zip(gpu[2:], caches[2:4]):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


def test_steps_that_follow_one_another():
    """Tables, write, prefill, decode and a block copy, 30 steps in a row without a look from the
    host, give what they give with the GPU waited for after each call."""
    n, hq, hkv, d, B, steps = 24, 8, 2, 128, 16, 30
    rng = np.random.default_rng(3)
    new = [rng.integers(1, 40, n)] + [rng.integers(0, 4, n) + (rng.random(n) < 0.1) * 20 for _ in range(steps - 1)]
    lens = np.cumsum(new, 0)
    T = -(-int(lens[-1].max()) // B)
    nb = int((-(-lens[-1] // B)).sum()) + 2
    inputs = []
    for q in new:
        rows = int(q.sum()) + 1
        inputs.append([dev16(rows16(rng, (rows, h, d), "bf16", 3), "bf16") for h in (hkv, hkv, hq)])
    outs = []
    for wait in (True, False):
        shape = (nb, hkv, B, d)
        caches = upload([np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8),
                         np.full(shape[:2], np.nan, np.float32), np.full(shape[:2], np.nan, np.float32)])
        tables = torch.full((n, T), -1, dtype=torch.int32, device="cuda")
        free, cells = dev(np.arange(nb - 1)[::-1], np.int32), [dev([0], np.int32), dev([0], np.int32)]
        slots = torch.empty(n * 60, dtype=torch.int64, device="cuda")
        c, q = [dev(x, np.int32) for x in lens], [dev(x, np.int32) for x in new]
        pair, got = dev([[1, nb - 1]], np.int32), []
        torch.cuda.synchronize()
        look = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(steps):
            key, value, query = inputs[i]
            qs, _ = pa.build_step(q[i], c[i], free, cells[i % 2], tables, B, nb, slots, free_next=cells[1 - i % 2])
            look()
            pa.append_fp8_block(key, value, *caches, tables, c[i], qs)
            look()
            got.append(pa.prefill_fp8_block(query, *caches, tables, c[i], qs, 0.1, int(new[i].max()))[:int(new[i].sum())])
            look()
            got.append(pa.decode_fp8_block(query[:n] if len(query) >= n else inputs[0][2][:n], *caches, tables, c[i], 0.1))
            look()
            pa.copy_blocks_fp8_block(*caches, pair)
            look()
        assert device_error() == 0
        outs.append(got + caches + [tables, slots])
    for a, b in zip(*outs):
        a, b = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in (a, b))
        assert torch.equal(a, b) or torch.equal(a.float().nan_to_num(7), b.float().nan_to_num(7))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_calls_with_nothing_to_do(dtype):
    b = Batch([20], 4, 2, 64, 16, "fp16", seed=1)
    caches = upload(b.written())
    before = [t.clone() for t in caches]
    i32 = dict(dtype=torch.int32, device="cuda")
    none, rows = torch.empty(0, **i32), torch.zeros(1, **i32)
    table = torch.empty(0, 4, **i32)
    kv, q = torch.empty(0, 2, 64, dtype=dtype, device="cuda"), torch.empty(0, 4, 64, dtype=dtype, device="cuda")
    pa.append_fp8_block(kv, kv, *caches, table, none, rows)
    pa.append_fp8_block(kv, kv, *caches, dev(b.tables), dev(b.ctx), torch.zeros(2, **i32))  # no new tokens
    pa.copy_blocks_fp8_block(*caches, torch.empty(0, 2, **i32))
    assert pa.decode_fp8_block(q, *caches, table, none, 0.1).shape == (0, 4, 64)
    assert pa.prefill_fp8_block(q, *caches, table, none, rows, 0.1, 0).shape == (0, 4, 64)
    slots = torch.full((3,), 9, dtype=torch.int64, device="cuda")
    qs, left = pa.build_step(none, none, torch.arange(5, **i32), dev([2], np.int32), table, 16, 9, slots)
    assert qs.tolist() == [0] and left.tolist() == [2] and slots.tolist() == [-1] * 3
    assert device_error() == 0 and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(caches, before))
