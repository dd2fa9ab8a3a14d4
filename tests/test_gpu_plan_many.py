"""GPU test of kq_kv_plan around the numbers of requests at which its block changes."""
import numpy as np
import pytest
import torch

import layerref as ref

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("R", [255, 256, 257, 1023, 1024, 1025, 1777, 2047, 2048, 2049, 4097, 8192])
@pytest.mark.parametrize("short", [False, True])
def test_plan(R, short):
    rng = np.random.default_rng(R)
    ps, width = 16, 8
    lens, add = rng.integers(0, 90, R), rng.integers(0, 30, R)
    held = -(-lens // ps)
    need = int((-(-(lens + add) // ps) - held).sum())
    perm = rng.permutation(int(held.sum()) + need + 5).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    free = perm[at:]
    n_free = need * 2 // 3 if short else len(free)
    T = int(add.sum()) + 3

    def d(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    plan, tab, status = kq.KVPlan(R, T), d(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    kq.kv_plan(d(lens), d(add), tab, d(free), d([n_free]), ps, plan, status=status)
    new, q_start, slots, pos, left, want, refused = ref.plan(lens.tolist(), add.tolist(), table.tolist(), free.tolist(), n_free,
                                                             ps, T)
    assert plan.lens.tolist() == new and plan.q_start.tolist() == q_start
    assert plan.slots.tolist() == slots and plan.pos.tolist() == pos
    assert plan.n_left.tolist() == [left] and tab.tolist() == [list(map(int, r)) for r in want]
    assert (status.item() != 0) == refused
