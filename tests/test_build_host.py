"""Host-only: the library needs neither torch nor a host C++ compiler; what the
Python marshalling of the layer operators needs costs only that module."""
import importlib.util
import os
import subprocess
import sys

import pytest

from gemv_nibble_unpack_amd import build as B


@pytest.fixture
def dry(tmp_path, monkeypatch):
    """A build into tmp_path whose commands are recorded and make empty files."""
    out = tmp_path / "lib.so"
    monkeypatch.setattr(B, "OUT", str(out))
    monkeypatch.setattr(B, "BIND_OUT", str(tmp_path / "bind.so"))
    monkeypatch.setattr(B, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(B, "undefined_kernels", lambda path: None)
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        if getattr(run, "refuse", None) and any(run.refuse in c for c in cmd):
            raise RuntimeError("refused")
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(B, "_run", run)
    return tmp_path, ran, run


def built(tmp_path):
    return sorted(p.name for p in tmp_path.iterdir() if p.suffix == ".so")


def test_all_is_built(dry):
    tmp, ran, _ = dry
    assert B.build(verbose=False) == B.OUT and built(tmp) == ["bind.so", "lib.so"]
    bind = [c for c in ran if B.BIND_SOURCE in c]
    assert len(bind) == 1
    # as torch says, not as assumed
    import torch
    assert f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}" in bind[0]


def test_library_without_torch(dry, monkeypatch, capsys):
    tmp, ran, _ = dry
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    (tmp / "bind.so").write_text("of another library")
    assert B.build(verbose=False) == B.OUT
    assert built(tmp) == ["lib.so"]                      # no marshalling of an older build either
    assert not any(B.BIND_SOURCE in c for c in ran)
    assert "torch" in capsys.readouterr().err


def test_library_without_host_compiler_or_python_headers(dry, monkeypatch, capsys):
    tmp, ran, _ = dry
    with monkeypatch.context() as m:
        m.setattr(B, "_cxx", lambda: None)
        assert B.build(verbose=False) == B.OUT and built(tmp) == ["lib.so"]
        assert "compiler" in capsys.readouterr().err
    with monkeypatch.context() as m:
        m.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp / "nowhere")})
        assert B.build(verbose=False) == B.OUT and built(tmp) == ["lib.so"]
        assert "Python.h" in capsys.readouterr().err


def test_broken_marshalling_is_an_error_behind_the_library(dry):
    tmp, _, run = dry
    run.refuse = B.BIND_SOURCE
    with pytest.raises(RuntimeError):
        B.build(verbose=False)
    assert built(tmp) == ["lib.so"]


def test_broken_library_is_an_error(dry):
    tmp, _, run = dry
    run.refuse = os.path.join(B.LAYER_CSRC, "norm.hip")
    with pytest.raises(RuntimeError):
        B.build(verbose=False)
    assert built(tmp) == []


def test_package_loads_its_library_without_the_marshalling():
    """The C library is loaded, and a layer operator says what is missing."""
    code = ("import sys; sys.modules['gemv_nibble_unpack_amd._layer_bind'] = None\n"
            "import gemv_nibble_unpack_amd as G\n"
            "G.load()\n"
            "try:\n    G.add_rmsnorm_q8(None, None)\n"
            "except G.LibraryMissing as e:\n    print('said', '_layer_bind' in str(e))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "said True" in r.stdout, r.stderr
