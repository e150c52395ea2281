"""The marshalling module belongs to the torch and the Python it was compiled against."""
import subprocess

import pytest

from selective_state_space_34_b200 import _abi, build


def test_marshalling_module_of_another_torch(monkeypatch):
    build.build()
    native = _abi.marshal()
    assert native.BUILT_FOR == build.built_for()
    ran = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: ran.append(cmd) or subprocess.CompletedProcess(cmd, 1, "", "stopped here"))
    build.build_marshal()
    assert not ran  # up to date
    monkeypatch.setattr(build, "built_for", lambda: "torch 0.1, another")
    with pytest.raises(RuntimeError, match="stopped here"):
        build.build_marshal()
    assert len(ran) == 1
    monkeypatch.setattr(_abi, "_native", None)
    with pytest.raises(ImportError, match="is built for torch"):
        _abi.marshal()
