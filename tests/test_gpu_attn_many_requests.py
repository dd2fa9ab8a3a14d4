"""GPU tests of kq_kv_attn for many query rows per key-value head and more requests
than its kernel keeps in shared memory."""
import numpy as np
import pytest
import torch

import test_gpu_attn as few

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("R,hi,window", [(1024, 90, 0), (1025, 90, 0), (3001, 70, 0), (1500, 300, 50)])
def test_many_requests_of_many_rows(kv, R, hi, window):
    rng = np.random.default_rng(R)
    counts = np.where(rng.random(R) < 0.1, 0, rng.integers(1, 3, R)).tolist()
    few.run(rng.integers(0, hi, R).tolist(), counts, 40, 1, 64, 16, kv, seed=R, max_q=2, window=window)
