"""GPU test: without the compiled fast path the layer operators' calls go through
ctypes and give the same results."""
import pytest
import torch

import layerref as ref

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def layer():
    """Every operator with its outputs given, as the fast path wants them: their results."""
    P = ref.Pool([40, 100], 2, 128, 16, "f16", seed=1, room=8)
    g = torch.Generator(device="cuda").manual_seed(2)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache, plan = kq.KVCache(torch.nan_to_num(P.k), torch.nan_to_num(P.v)), kq.KVPlan(2, 4)
    table = P.table_dev.contiguous()
    kq.kv_plan(torch.tensor([40, 100], **i32), torch.tensor([1, 3], **i32), table, torch.from_numpy(P.free).cuda(),
               torch.tensor([len(P.free)], **i32), 16, plan)
    qkv = torch.randn(4, 12 * 128, generator=g, device="cuda")
    q, a = torch.empty(4, 8 * 128, device="cuda"), torch.empty(4, 8 * 128, device="cuda")
    kq.kv_append(qkv, 8, cache, plan.slots, plan.pos, torch.rand(64, generator=g, device="cuda"), q_out=q)
    ws = torch.empty(kq.kv_attn_workspace_bytes(2, 3, 8, cache), dtype=torch.uint8, device="cuda")
    kq.kv_attn(q, cache, plan.lens, table, q_start=plan.q_start, max_q=3, out=a, workspace=ws)
    out, h = torch.empty_like(a), torch.empty_like(a)
    kq.residual_norm(q, a, pre_gamma=torch.ones(1024, device="cuda"), out=out, h=h)
    return [plan.lens, plan.q_start, plan.slots, plan.pos, plan.n_left, table, q, cache.k, cache.v, a, out, h]


def test_results_are_the_same(monkeypatch):
    fast = layer()
    monkeypatch.setattr(kq, "_fast", kq._NoFastPath)
    slow = layer()
    assert all(torch.equal(x, y) for x, y in zip(fast, slow))
