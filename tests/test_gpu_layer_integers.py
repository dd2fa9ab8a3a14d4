"""GPU tests: whole numbers that do not fit the C ABI's 32 bits are refused by
the binding of the layer operators (ctypes alone would cut them)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")
BIG = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kw", [dict(window=BIG + 5), dict(window=1 << 31), dict(window=-BIG), dict(max_q=BIG + 1), dict(max_q=BIG)])
def test_attention(kw, given):
    k = torch.randn(3, 1, 16, 64, device="cuda").half()
    cache, q = kq.KVCache(k, k.clone()), torch.randn(1, 64, device="cuda")
    more = dict(out=torch.empty_like(q), workspace=torch.empty(kq.kv_attn_workspace_bytes(1, 1, 1, cache), dtype=torch.uint8,
                                                               device="cuda")) if given else {}
    with pytest.raises(ValueError, match=next(iter(kw))):
        kq.kv_attn(q, cache, i32(40), i32(0, 1, 2).view(1, 3), **kw, **more)


@pytest.mark.parametrize("R,max_q,n_q,name", [(BIG + 1, 1, 1, "R"), (1, BIG + 1, 1, "max_q"), (1, 1, BIG + 1, "n_q")])
def test_workspace(R, max_q, n_q, name):
    k = torch.zeros(3, 1, 16, 64, device="cuda").half()
    with pytest.raises(ValueError, match=name):
        kq.kv_attn_workspace_bytes(R, max_q, n_q, kq.KVCache(k, k))


def test_plan():
    with pytest.raises(ValueError, match="page_size"):
        kq.kv_plan(i32(3), i32(1), i32(0, -1).view(1, 2), i32(1, 2), i32(2), BIG + 16, kq.KVPlan(1, 1))
