"""Values at the ends of their range that the layer operators refuse on the
host, before a device is touched.  Skipped where there is a GPU, as
test_host_layer_ops (whose stand-in calls are used) is."""
import pytest
import torch

import test_host_layer_ops as ops

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks")


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_attention_refuses_a_scale_beyond_fp32_in_powers_of_two(scale):
    """scale is finite, scale * log2(e), which the scores are taken with, is not."""
    assert ops.attn(scale=scale) == ops.INVALID
    assert b"scale" in ops.kq.lib().kq_last_error()


def test_an_empty_residual_step_needs_no_arrays():
    """An empty tensor's address is NULL."""
    none = dict(y=None, res=None, out=None, h=None, pre_gamma=None)
    assert ops.residual(T=0, **none) == 0 and ops.residual(N=0, **none) == 0
    assert ops.residual(**none) == ops.INVALID
