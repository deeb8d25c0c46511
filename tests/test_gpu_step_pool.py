"""The GPU's step planning on top of the host pool: the blocks that steps hand out are a reserve that
the pool holds under an id of its own, so that one ledger knows every block."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from fp8_block_harness import dev
from gpu_harness import device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def test_a_reserve_of_the_pool_feeds_the_steps():
    """Prompts placed by the pool, decode steps planned on the GPU from a reserve: no block has two
    owners, what the steps took can be told from free_next, and the pool gets all of it back."""
    B, nb, T, n, reserve = 16, 64, 12, 4, 1000
    pool = pa.BlockPool(nb, B)
    lens = np.array([20, 16, 45, 1])
    tables = np.full((n, T), -1, np.int32)
    for s in range(n):
        pool.allocate(s, int(lens[s]))
        t = pool.block_table(s)
        tables[s, :len(t)] = t
    pool.allocate(reserve, 20 * B)
    stock = np.asarray(pool.block_table(reserve), np.int32)
    assert len(stock) == 20 and not np.isin(stock, tables).any()
    gt, free, cells = dev(tables), dev(stock), [dev([0], np.int32), dev([0], np.int32)]
    slots, ones = torch.empty(n, dtype=torch.int64, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    for i in range(60):
        pa.build_step(ones, dev(lens + i + 1, np.int32), free, cells[i % 2], gt, B, nb, slots, free_next=cells[1 - i % 2])
        if i == 30:  # a request that comes in meanwhile is placed by the pool, beside the reserve
            pool.allocate(77, 40)
    assert device_error() == 0
    got, used = gt.cpu().numpy(), int(cells[0])
    need = -(-(lens + 60) // B)
    owned = np.concatenate([got[s, :need[s]] for s in range(n)] + [pool.block_table(77)])
    assert len(set(owned.tolist())) == len(owned) and (got[np.arange(T)[None] >= need[:, None]] == -1).all()
    assert used == need.sum() - (-(-lens // B)).sum()
    np.testing.assert_array_equal(np.sort(stock[:used]), np.sort(np.setdiff1d(owned, np.concatenate([tables.ravel(), pool.block_table(77)]))))
    for s in [*range(n), reserve, 77]:
        pool.free(s)
    assert pool.num_free() == nb
