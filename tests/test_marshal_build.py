"""The compiled marshalling is loaded only where it was built for the running Python and torch (CPU)."""
import os

import pytest


@pytest.fixture()
def vh(monkeypatch):
    import verify_head_gb300 as vh
    vh.build()
    monkeypatch.setattr(vh, "_compiled", None)
    return vh


def test_built_and_bound(vh):
    from verify_head_gb300 import buildlib
    path = buildlib.build_marshal()
    if path is None:
        pytest.skip("the marshalling cannot be compiled here")
    assert os.path.exists(path)
    m = vh._compiled_calls()
    assert m and m.add_rmsnorm() == 1  # not the usual kind of call: left to the binding's own checks
    assert m.__file__ == path


@pytest.mark.parametrize("what", ["torch", "build of torch", "python"])
def test_other_versions_are_not_loaded(vh, monkeypatch, what):
    import sysconfig

    import torch
    from verify_head_gb300 import buildlib
    before = buildlib.marshal_path()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "99.0.0+none")
    elif what == "build of torch":
        monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
    else:
        real = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda k: "cpython-99-none" if k == "SOABI" else real(k))
    assert buildlib.marshal_path() != before and os.path.exists(buildlib.marshal_path()) is False
    assert vh._compiled_calls() is False
