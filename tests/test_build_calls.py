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


def test_a_failed_kernel_leaves_no_child_behind(monkeypatch, tmp_path):
    """_calls.so is compiled beside the kernels: it is waited for when one of them fails."""
    child = Child()
    tmp = tmp_path / "_calls.so.tmp"
    tmp.write_bytes(b"made")
    monkeypatch.setattr(build, "build_calls", lambda force=False: (child, str(tmp)))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "sources", lambda: [str(tmp_path / "none.cu")])
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(force=True)
    assert child.collected and not tmp.exists()


def test_a_failed_one_leaves_no_temporary_file(monkeypatch, tmp_path):
    child = Child()
    child.returncode = 1
    tmp = tmp_path / "_calls.so.tmp"
    tmp.write_bytes(b"half of it")
    with pytest.raises(RuntimeError, match="kq_calls.cpp"):
        build.finish_calls((child, str(tmp)))
    assert not tmp.exists()


def test_without_torchs_headers_it_is_left_out(monkeypatch, tmp_path, capsys):
    """The library needs neither torch's headers nor g++."""
    import torch.utils.cpp_extension as ext
    monkeypatch.setattr(build.subprocess, "Popen", Child)
    monkeypatch.setattr(ext, "include_paths", lambda *a, **k: [str(tmp_path)])
    assert build.build_calls(force=True) is None
    assert "python_variable.h" in capsys.readouterr().out


def test_without_a_compiler_it_is_left_out(monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(build.subprocess, "Popen", Child)
    monkeypatch.setenv("PATH", str(tmp_path))
    assert build.build_calls(force=True) is None
    assert "g++" in capsys.readouterr().out
