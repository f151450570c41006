"""What build() makes and when: the library by itself, and the compiled half of
the Python binding for the torch that is installed."""
import os
import subprocess
import sys

import pytest
import torch

from weight_only_quantized_wql_gb300 import _build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A source tree of one kernel and a binding that does not compile."""
    csrc, out = tmp_path / "csrc", tmp_path / "_build"
    csrc.mkdir()
    out.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (csrc / "binding.cpp").write_text("#error no headers here\n")
    for name, value in (("CSRC", csrc), ("BUILD", out), ("LIB", out / "libwql.so"),
                        ("BINDING", out / "_wql_torch.so"), ("BINDING_SRC", csrc / "binding.cpp"),
                        ("BINDING_FOR", out / "_wql_torch.for")):
        monkeypatch.setattr(_build, name, str(value))
    return out


def test_library_is_built_when_the_binding_cannot_be(small):
    with pytest.raises(RuntimeError, match="no headers here"):
        _build.build()
    assert os.path.exists(_build.LIB) and _build.library_up_to_date()
    assert not _build.up_to_date()
    t = os.path.getmtime(_build.LIB)
    assert _build.build(binding=False) == _build.LIB          # nothing left to do
    assert os.path.getmtime(_build.LIB) == t


def test_binding_belongs_to_a_torch_and_a_python(small, monkeypatch):
    for path, text in ((_build.LIB, ""), (_build.BINDING, ""), (_build.BINDING_FOR, _build._built_for())):
        with open(path, "w") as f:
            f.write(text)
    assert _build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.1")
        assert _build.library_up_to_date() and not _build.up_to_date()
    os.remove(_build.BINDING_FOR)
    assert not _build.up_to_date()


def test_library_needs_no_torch(small):
    """The build file by itself, in a Python that cannot import torch."""
    code = (f"import sys; sys.modules['torch'] = None; sys.path.insert(0, {os.path.dirname(_build.__file__)!r})\n"
            "import _build, os\n" +
            "".join(f"_build.{n} = {getattr(_build, n)!r}\n"
                    for n in ("CSRC", "BUILD", "LIB", "BINDING", "BINDING_SRC", "BINDING_FOR")) +
            "_build.build(binding=False)\nassert os.path.exists(_build.LIB)\n"
            "os.remove(_build.LIB)\n"
            "try:\n    _build.build()\nexcept ImportError:\n    pass\n"
            "assert os.path.exists(_build.LIB)\n")
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
