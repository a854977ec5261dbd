"""Where the compiled module of the serving calls cannot be built (no Python headers), the library is built all the same:
its other calls do not need it."""
import os

import pytest

from gather_radix_select_gb300 import build


@pytest.fixture
def without_headers(monkeypatch, tmp_path):
    """A build in a folder of its own, whose library is a stand-in and whose compiler finds no headers."""
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "build", lambda force=False, debug=False, **_: "debug" if debug else "release")
    monkeypatch.setenv("CXX", "/bin/false")


def test_the_library_is_built_where_the_module_cannot_be(without_headers):
    with pytest.warns(RuntimeWarning, match="cache_append"):
        assert build.build_all(force=True) == ["release", "debug"]


def test_no_module_of_an_earlier_build_is_left(without_headers):
    # (it would be called with the library that was just built)
    so = build.binding_path()
    os.makedirs(os.path.dirname(so))
    open(so, "w").close()
    with pytest.warns(RuntimeWarning):
        build.build_all(force=True)
    assert not os.path.exists(so)


def test_calls_that_need_the_module_say_so(without_headers, monkeypatch):
    from gather_radix_select_gb300 import _native
    monkeypatch.setattr(_native, "_binding", None)
    monkeypatch.setattr(_native, "load", lambda: None)
    with pytest.raises(RuntimeError, match="not built"):
        _native.binding()
