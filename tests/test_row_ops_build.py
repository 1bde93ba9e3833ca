"""The extension module of the row operators belongs to one torch and one Python:
built for others it is compiled again, and refused rather than loaded."""
import pytest

from logits_sampling_gb300 import _row_ops, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_a_built_extension_is_up_to_date():
    assert build._binding_up_to_date()


@pytest.mark.parametrize("was", [None, "", "torch 1.0.0, cpython-312\n"])
def test_an_extension_for_another_torch_is_neither_kept_nor_loaded(monkeypatch, tmp_path, was):
    note = tmp_path / "for"
    if was is not None:
        note.write_text(was)
    monkeypatch.setattr(build, "BINDING_FOR", str(note), raising=False)
    assert not build._binding_up_to_date()
    monkeypatch.setattr(_row_ops, "_calls", None)
    with pytest.raises(RuntimeError, match="run `python -m logits_sampling_gb300.build`"):
        _row_ops.calls()


def test_another_torch_asks_for_another_build(monkeypatch):
    import importlib.metadata
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "1.0.0")
    assert not build._binding_up_to_date()
    monkeypatch.setattr(_row_ops, "_calls", None)
    with pytest.raises(RuntimeError, match="this is torch 1.0.0"):
        _row_ops.calls()
