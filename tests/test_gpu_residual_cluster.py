"""GPU tests of kq_residual_norm where a column is split over a cluster's
blocks, beside work on another stream that keeps the multiprocessors busy, so
that a cluster's blocks begin and reach their sums at different times: sizes
from two to eight blocks per column, none, one or both of the norms."""
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


@pytest.mark.parametrize("T,N", [(1, 1025), (1, 2048), (1, 4096), (3, 4097), (9, 8192), (18, 5000), (37, 2050), (1, 131072)])
@pytest.mark.parametrize("post,pre", [(False, False), (False, True), (True, False), (True, True)])
def test_blocks_that_begin_at_different_times(T, N, post, pre):
    rng = np.random.default_rng(T + N)

    def f(*s):
        return rng.standard_normal(s).astype(np.float32)
    res, y = f(T, N), f(T, 2, N)
    w, pg, qg = np.abs(f(T, 2)), (1 + 0.2 * f(N) if post else None), (1 + 0.2 * f(N) if pre else None)
    d = [None if x is None else torch.from_numpy(x).cuda() for x in (res, y, w, pg, qg)]
    o, h, eo, eh = ref.residual(res, y, w, pg, None, 0.7, qg, 1e-5)
    busy = torch.randn(1 << 22, device="cuda")
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(other):
        for _ in range(60):
            busy = torch.sin(busy)
    with torch.cuda.stream(mine):
        for _ in range(40):
            got.append(kq.residual_norm(d[0], d[1], weights=d[2], post_gamma=d[3], scale=0.7, pre_gamma=d[4], eps=1e-5))
    torch.cuda.synchronize()
    ref.check(got[0][0], o, eo + 1e-37, "out")
    if pre:
        ref.check(got[0][1], h, eh + 1e-37, "h")
    for a, b in got[1:]:
        assert torch.equal(a, got[0][0]) and (not pre or torch.equal(b, got[0][1]))
