"""The build and the loading of _calls.so, the binding's fast path, on the CPU."""
import sys

import pytest
import torch

from dequant_quant_gemv_b200 import build

build.build()


class Child:
    """A g++ that is not run."""
    returncode, collected = 0, False

    def __init__(self, cmd=None, **kw):
        self.cmd = cmd

    def communicate(self):
        self.collected = True
        return b"", None


def test_an_up_to_date_one_is_kept():
    assert build.build_calls() is None


def test_another_torch_needs_another_one(monkeypatch):
    monkeypatch.setattr(build.subprocess, "Popen", Child)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    started = build.build_calls()
    assert started is not None and started[0].cmd[0] == "g++"


@pytest.mark.filterwarnings("ignore:_calls.so")
def test_one_of_another_torch_is_not_taken(monkeypatch):
    kq = pytest.importorskip("dequant_quant_gemv_b200.kq")
    monkeypatch.setattr(kq, "_layer", None)
    monkeypatch.setattr(kq, "_fast", None)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    try:
        kq._layer_lib()
    except ImportError:
        pass
    from dequant_quant_gemv_b200 import _calls
    assert kq._fast is not _calls


def test_the_operators_work_without_it(monkeypatch):
    kq = pytest.importorskip("dequant_quant_gemv_b200.kq")
    monkeypatch.setattr(kq, "_layer", None)
    monkeypatch.setattr(kq, "_fast", None)
    monkeypatch.setitem(sys.modules, "dequant_quant_gemv_b200._calls", None)  # its import fails
    monkeypatch.delattr(sys.modules["dequant_quant_gemv_b200"], "_calls", raising=False)
    with pytest.warns(RuntimeWarning, match="_calls.so"):
        assert kq._layer_lib().kq_residual_norm(None, 1, 64, None) == 1
    x, g = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError):  # the checks in Python
        kq.residual_norm(x, x, pre_gamma=g, out=x.clone(), h=x.clone())
