"""CPU tests of when the library and the compiled binding are built again."""

import pytest

from paged_kv_gb300 import build


def test_nothing_to_do_after_a_build():
    build.build()
    assert not build.stale()


@pytest.mark.parametrize("what", ["version", "place"])
def test_another_torch_makes_the_binding_stale(monkeypatch, what):
    """It is compiled against one torch's headers and linked to its libraries."""
    build.build()
    if what == "version":
        real = build.importlib.metadata.version
        monkeypatch.setattr(build.importlib.metadata, "version",
                            lambda name: "0.0" if name == "torch" else real(name))
    else:
        monkeypatch.setattr(build, "_torch_dir", lambda: "/elsewhere/torch")
    assert build.stale()


def test_a_build_that_recorded_no_torch_is_stale(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "none"))
    assert build.stale()
