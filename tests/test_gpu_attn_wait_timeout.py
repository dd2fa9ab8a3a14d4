"""Failure detection in the attention kernel for many rows: a bounded wait that
runs out.

Its warps hand each other chunks through barriers.  The test hook
kq_inject("hold_attn@N") withholds one hand-over of the first block and shortens
the limit of the waits to 1 ms.  The launch ends, the host reads the fault
word, other blocks' results stay right, and the context stays usable."""
import numpy as np
import pytest
import torch

import layerref as ref
import test_gpu_attn as few

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")
KQ_ERR_TIMEOUT = 6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.device_fault()          # start from a clear fault word
    yield
    kq.inject(None)


@pytest.mark.parametrize("kv,D", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("hold", [1, 2, 3, 4, 6])
def test_a_withheld_chunk_times_out_and_the_context_survives(kv, D, hold):
    """4 requests of 2000 keys and 8 key-value heads: 6 chunks for the first block."""
    n, cols, n_kv, n_q = 2000, 8, 8, 128
    P = ref.Pool([n] * 4, n_kv, D, 16, kv, seed=D)
    q, dq = few.queries(4 * cols, n_q * D, 5)
    cache, lens, qs = kq.KVCache(P.k, P.v), few.i32([n] * 4), few.i32(np.arange(5) * cols)
    ws = torch.empty(kq.kv_attn_workspace_bytes(4, cols, n_q, cache), dtype=torch.uint8, device="cuda")

    def call():
        return kq.kv_attn(dq, cache, lens, P.table_dev, q_start=qs, max_q=cols, workspace=ws)
    want = call()
    torch.cuda.synchronize()                     # nothing queued ahead of the launch
    assert kq.device_fault() == 0
    kq.inject(f"hold_attn@{hold}")
    late = call()
    torch.cuda.synchronize()                     # the launch ends: no hang
    assert kq.device_fault() == KQ_ERR_TIMEOUT
    assert kq.device_fault() == 0                # read and cleared
    assert torch.equal(late[cols:], want[cols:])  # (the first block has keys of the first request only)
    # the hook was one-shot and the context is intact
    assert torch.equal(call(), want)
    torch.cuda.synchronize()
    assert kq.device_fault() == 0


def test_calls_of_few_rows_leave_the_hook_for_the_next_of_many():
    P = ref.Pool([20000], 1, 64, 64, "f16", seed=1)  # (long enough for a chunk in the first block)
    cache, lens = kq.KVCache(P.k, P.v), few.i32([20000])
    kq.inject("hold_attn@1")
    kq.kv_attn(few.queries(1, 64, 2)[1], cache, lens, P.table_dev)
    assert kq.device_fault() == 0
    kq.kv_attn(few.queries(1, 100 * 64, 3)[1], cache, lens, P.table_dev)
    assert kq.device_fault() == KQ_ERR_TIMEOUT
    kq.inject("hold_attn@1")
    kq.inject(None)
    kq.kv_attn(few.queries(1, 100 * 64, 3)[1], cache, lens, P.table_dev)
    assert kq.device_fault() == 0


def test_inject_rejects_unknown_specs():
    for spec in ("hold_attn@0", "hold_attn@", "hold_attn@-1", "hold_attn@1x", "hold_attn"):
        with pytest.raises(kq.KQError):
            kq.inject(spec)
    kq.inject(None)
