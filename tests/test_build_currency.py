"""When the build counts as current: the extension module is tied to one Python and one torch."""

import importlib.metadata
import os

from virtual_noise_perturbed_gb300 import build as b


def test_an_upgrade_of_torch_or_python_rebuilds_the_extension(monkeypatch):
    b.build()
    assert b.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "0.0.0")
        assert not b.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399")
        assert not b.up_to_date()
    assert b.up_to_date()


def test_an_interrupted_link_is_not_current(monkeypatch, tmp_path):
    """The record is written last: without it, or with that of another build, the libraries are not taken."""
    b.build()
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    assert not b.up_to_date()
    with open(os.path.join(tmp_path, "binding.made_for"), "w") as f:
        f.write("another")
    assert not b.up_to_date()
