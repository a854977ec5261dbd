"""The compiled module of the serving calls: its file goes with the interpreter and with PyTorch."""
import sysconfig

from gather_radix_select_gb300 import build


def test_the_file_goes_with_the_interpreter_and_with_pytorch(monkeypatch):
    import torch
    here = build.binding_path()
    own = sysconfig.get_config_var
    assert own("SOABI")
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other" if name == "SOABI" else own(name))
    other = build.binding_path()
    assert other != here
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert build.binding_path() not in (here, other)
