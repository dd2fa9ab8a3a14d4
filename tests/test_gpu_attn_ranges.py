"""GPU tests of kq_kv_attn where scores and queries are as large as fp32
allows.  1, 9, 24 and 100 query heads per key-value head reach each of the
kernels."""
import numpy as np
import pytest
import torch

import layerref as ref

pytestmark = pytest.mark.gpu
kq = pytest.importorskip("dequant_quant_gemv_b200.kq")
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def call(kv, D, n_q, n, keys, size):
    """One request of n tokens; dimension 7 of the keys holds `keys`, all else 0;
    dimension 7 of every query is such that a key of 1 has the score `size` in
    powers of two.  (out (n_q, D), the values (n, D))."""
    P = ref.Pool([n], 1, D, 16, kv, seed=n_q)
    P.k.mul_(0.0)
    pages = P.table[0]
    for i, x in enumerate(keys):
        if x:
            P.k[pages[i // 16], 0, i % 16, 7] = x
    q = torch.zeros(1, n_q, D, device="cuda")
    q[:, :, 7] = size / LOG2E
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = kq.kv_attn(q.view(1, -1), kq.KVCache(P.k, P.v), lens, P.table_dev, scale=1.0)
    return out.view(n_q, D), P.rows(P.v, 0, 0, n)


def check(out, V, want):
    # The weights are 0, 1 or powers of two, whatever the scores' size, so the
    # sum over n equal weights is exact and the mean has the roundings of at
    # most 64 additions per part and the joins (U each) and of the division.
    bound = 96 * ref.U * np.abs(V).mean(0) + 4 * ref.U * np.abs(want) + 1e-37
    ref.check(out, np.broadcast_to(want, out.shape), np.broadcast_to(bound, out.shape), "out")


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("n_q,D", [(1, 64), (9, 128), (24, 64), (100, 128)])
@pytest.mark.parametrize("size", [2.0 ** 126 * 1.5, 2.0 ** 127, 2.0 ** 127 * 1.7])
def test_queries_of_the_largest_binade(kv, n_q, D, size):
    n = 70
    for sign in (1.0, -1.0):
        keys = np.zeros(n)
        keys[20] = 1.0
        out, V = call(kv, D, n_q, n, keys, sign * size)
        check(out, V, V[20] if sign > 0 else np.delete(V, 20, 0).mean(0))


LARGE = [2.0 ** 24 - 3, 2.0 ** 25 + 4, 2.0 ** 25 + 12, 2.0 ** 26 + 8, 1e8, 2e8, 2.0 ** 28 + 32, 3e9]


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("n_q,D", [(1, 64), (9, 64), (24, 128), (100, 64)])
@pytest.mark.parametrize("size", LARGE)
def test_scores_whose_step_is_large(kv, n_q, D, size):
    """Equal scores weigh the same whatever their size; of unequal ones the largest has all."""
    n = 90
    out, V = call(kv, D, n_q, n, np.ones(n), size)
    check(out, V, V.mean(0))
    out, V = call(kv, D, n_q, n, np.ones(n), -size)
    check(out, V, V.mean(0))
    keys = np.full(n, 0.5)
    keys[61] = 1.0
    out, V = call(kv, D, n_q, n, keys, size)
    check(out, V, V[61])
    out, V = call(kv, D, n_q, n, keys, -size)
    check(out, V, np.delete(V, 61, 0).mean(0))


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("n_q", [1, 100])
@pytest.mark.parametrize("size", [2.0 ** 25 + 4, 1e8, 2e8])
def test_large_scores_over_many_blocks(kv, n_q, size):
    """Parts with maxima of every size are joined."""
    n = 5000
    keys = np.zeros(n)
    keys[3000], keys[3100] = 1.0, 1.0
    out, V = call(kv, 64, n_q, n, keys, size)
    check(out, V, (V[3000] + V[3100]) / 2)


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("n_q,D", [(1, 64), (9, 64), (24, 128), (100, 64)])
@pytest.mark.parametrize("n", [50, 2000])
def test_scores_at_the_end_of_the_range(kv, n_q, D, n):
    """Finite scores between -3e38 and the lowest fp32 value are scores, too."""
    for size in (-2.9e38, -3.05e38, -3.3e38, 3.3e38):
        out, V = call(kv, D, n_q, n, np.ones(n), size)
        check(out, V, V.mean(0))
