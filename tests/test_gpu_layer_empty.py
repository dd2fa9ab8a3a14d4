"""GPU tests: calls of the layer operators with nothing to do (no columns, no
requests, no rows, no free pages) leave everything as it is."""
import pytest
import torch

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,N", [(0, 640), (3, 0), (0, 0)])
def test_residual(T, N):
    x, g = torch.empty(T, N, device="cuda"), torch.empty(N, device="cuda")
    for kw in (dict(), dict(out=torch.empty_like(x), h=torch.empty_like(x))):
        out, h = kq.residual_norm(x, x.clone(), post_gamma=g, pre_gamma=g, **kw)
        assert out.shape == h.shape == (T, N)


def test_residual_without_rows():
    x = torch.randn(7, 640, device="cuda")
    assert torch.equal(kq.residual_norm(x, torch.empty(7, 0, 640, device="cuda"))[0], x)


def test_append_and_attention():
    k = torch.randn(3, 1, 16, 64, device="cuda").half()
    cache = kq.KVCache(k, k.clone())
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert kq.kv_append(torch.empty(0, 4 * 64, device="cuda"), 2, cache, none, i32(), None).shape == (0, 128)
    q = torch.empty(0, 128, device="cuda")
    assert kq.kv_attn(q, cache, i32(), torch.empty(0, 3, dtype=torch.int32, device="cuda")).shape == (0, 128)
    assert kq.kv_attn(q, cache, i32(5), i32(0, 1).view(1, 2), q_start=i32(0, 0)).shape == (0, 128)
    # columns of no request
    out = torch.full((2, 128), 7.0, device="cuda")
    kq.kv_attn(torch.randn(2, 128, device="cuda"), cache, i32(5), i32(0, 1).view(1, 2), q_start=i32(1, 1), out=out)
    assert (out == 7.0).all()


def test_plan():
    p = kq.kv_plan(i32(), i32(), torch.empty(0, 4, dtype=torch.int32, device="cuda"), i32(1, 2), i32(2), 16, kq.KVPlan(0, 3))
    assert p.slots.tolist() == p.pos.tolist() == [-1] * 3 and p.q_start.tolist() == [0] and p.n_left.tolist() == [2]
    table = i32(0, -1, 1, -1).view(2, 2)
    p = kq.kv_plan(i32(3, 4), i32(0, 0), table, i32(), i32(0), 16, kq.KVPlan(2, 0))
    assert p.lens.tolist() == [3, 4] and p.q_start.tolist() == [0, 0, 0] and p.n_left.tolist() == [0]
    assert table.tolist() == [[0, -1], [1, -1]]
