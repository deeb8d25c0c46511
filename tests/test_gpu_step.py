"""build_step on the GPU against its definition: tables, slots, offsets and the list's next
cell are equal, entries that a step does not own stay as they were, and a step that cannot be
served changes nothing."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from gpu_harness import device_error
from oracle import fp8_block as fb

pytestmark = pytest.mark.gpu

BITS = {"blocks": pa.DEVERR_NO_BLOCKS, "slots": pa.DEVERR_BAD_SLOT, "context": pa.DEVERR_BAD_CONTEXT,
        "block": pa.DEVERR_BAD_BLOCK}


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.array(x, dtype=dtype)).cuda()


def check(new, past, B, T, spare=3, pad=5, start=2, seed=0, free=None, num_blocks=None, tables=None,
          slots=None):
    rng = np.random.default_rng(seed)
    new, ctx = np.array(new, np.int64), np.array(new, np.int64) + np.array(past, np.int64)
    have, need = -(-np.array(past) // B), -(-ctx // B) - -(-np.array(past) // B)
    nb = int(have.sum() + max(need.sum(), 0) + start + spare) + 1 if num_blocks is None else num_blocks
    order = rng.permutation(nb).astype(np.int32)
    if tables is None:
        tables, at = np.full((len(new), T), -9, np.int32), 0
        for s, h in enumerate(have):
            tables[s, :h] = order[at:at + h]
            at += h
        order = order[at:]
    if free is None:
        free = order[:start + int(need.sum()) + spare]
    n_slots = int(new.clip(0).sum()) + pad if slots is None else slots
    want = fb.build_step(new, ctx, free, start, tables, B, nb, n_slots)
    t = dev(tables)
    slot_mapping = torch.full((n_slots,), -77, dtype=torch.int64, device="cuda")
    qs, nxt = pa.build_step(dev(new), dev(ctx), dev(free), dev([start]), t, B, nb, slot_mapping)
    assert device_error() == sum(BITS[e] for e in want[4])
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(slot_mapping.cpu().numpy(), want[1])
    np.testing.assert_array_equal(qs.cpu().numpy(), want[2])
    assert nxt.item() == want[3]
    return want


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("n", [1, 2, 33, 255, 256, 257, 700])
def test_mixed_batches(n, B):
    rng = np.random.default_rng(n * 100 + B)
    kind = rng.integers(0, 4, n)
    new = np.where(kind == 0, 1, np.where(kind == 1, 0, rng.integers(1, 150, n)))
    past = np.where(kind == 3, 0, rng.integers(0, 200, n))
    assert not check(new, past, B, 1 + 350 // B, seed=n)[4]


@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [15]), ([1], [16]), ([16], [0]), ([17], [15]),
                                      ([0], [0]), ([0, 0, 5, 0], [3, 0, 16, 16]), ([5000], [3])])
def test_edges(new, past):
    assert not check(new, past, 16, 320)[4]


def test_more_slots_than_one_pass_of_the_grid():
    assert not check([200000, 1, 450000], [3, 40, 0], 16, 30000, pad=100000)[4]


def test_no_sequences():
    tables = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    slots = torch.zeros(7, dtype=torch.int64, device="cuda")
    qs, nxt = pa.build_step(none, none, dev([1, 2]), dev([1]), tables, 16, 8, slots)
    assert qs.tolist() == [0] and nxt.item() == 1 and slots.tolist() == [-1] * 7 and device_error() == 0


@pytest.mark.parametrize("kw,err", [
    (dict(new=[40, 8], past=[0, 3], spare=-1), {"blocks"}),
    (dict(new=[40, 8], past=[0, 3], free=np.arange(9), start=10), {"blocks"}),
    (dict(new=[40, 8], past=[0, 3], free=np.arange(9), start=-1, num_blocks=20), {"blocks"}),
    (dict(new=[40, 8], past=[0, 3], slots=47), {"slots"}),
    (dict(new=[40, 8], past=[0, 3], slots=0, spare=-1), {"blocks", "slots"}),
    (dict(new=[5, -3, 9, 4], past=[0, 9, -4, 16 * 6], T=6, num_blocks=40), {"context"}),
    (dict(new=[20, 8], past=[0, 3], free=np.array([3, 99, -1, 5, 6, 7]), start=0, num_blocks=9), {"block"}),
    (dict(new=[20, 2], past=[3, 14], tables=np.array([[12, -1, -1], [-5, 1, 1]], np.int32),
          free=np.array([3, 4, 5]), start=0, num_blocks=9), {"block"}),
])
def test_steps_that_cannot_be_served(kw, err):
    got = check(**{"B": 16, "T": kw.get("tables", np.zeros((0, 6))).shape[1], **kw})[4]
    assert got == err


def test_captured_steps_follow_one_another():
    """Two decode steps planned from one graph, replayed with lengths that the graph itself
    raises: the list's next cell feeds the following step."""
    B, n, T = 8, 5, 6
    past = np.array([7, 8, 15, 1, 0])
    order = np.random.default_rng(1).permutation(40).astype(np.int32)
    have = -(-past // B)
    tables, at = np.full((n, T), -1, np.int32), 0
    for s, h in enumerate(have):
        tables[s, :h] = order[at:at + h]
        at += h
    free = order[at:]
    one, ctx = dev(np.ones(n)), dev(past)
    t, cells, f = dev(tables), [dev([0]), dev([0])], dev(free)
    qs = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    slots = [torch.zeros(n + 1, dtype=torch.int64, device="cuda") for _ in range(2)]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            for k in range(2):
                ctx += 1
                pa.build_step(one, ctx, f, cells[k], t, B, 40, slots[k], qs, cells[1 - k])
    torch.cuda.synchronize()
    wt, start = tables, 0
    for r in range(4):
        g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            past = past + 1
            wt, ws, _, start, errs = fb.build_step(np.ones(n), past, free, start, wt, B, 40, n + 1)
            assert not errs
            np.testing.assert_array_equal(slots[k].cpu().numpy(), ws)
        np.testing.assert_array_equal(t.cpu().numpy(), wt)
        assert cells[0].item() == start
    assert device_error() == 0


def test_another_stream():
    s = torch.cuda.Stream()
    q, c = dev([20, 1]), dev([20, 17])
    t, slots = dev([[0, 0], [5, 0]]), torch.zeros(22, dtype=torch.int64, device="cuda")
    f, start = dev([7, 8, 9]), dev([0])
    s.wait_stream(torch.cuda.current_stream())
    qs, nxt = pa.build_step(q, c, f, start, t, 16, 10, slots, stream=s)
    s.synchronize()
    assert t.tolist() == [[7, 8], [5, 9]] and nxt.item() == 3 and qs.tolist() == [0, 20, 21]
    assert slots.tolist() == [*range(112, 128), *range(128, 132), 9 * 16, -1]
