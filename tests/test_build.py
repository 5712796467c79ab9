"""What each of the two builds needs and notices (nothing is compiled here)."""
import os

import pytest

from gated_delta_rule_gate_gb300 import build as b


@pytest.fixture
def nothing_runs(monkeypatch):
    def refuse(cmd, **kw):
        raise AssertionError("ran %s" % cmd[0])
    monkeypatch.setattr(b.subprocess, "run", refuse)


def test_the_library_needs_no_binding(monkeypatch, nothing_runs, tmp_path):
    """Without g++, torch or a binding the library is up to date, and stays."""
    b.build()
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "none.so"))
    assert b.up_to_date() and b.build() == b.LIB


def test_a_failing_binding_leaves_the_library(monkeypatch, tmp_path):
    """Both builds at once: the library is there when the error of the other comes."""
    made = []
    monkeypatch.setattr(b, "build", lambda **kw: made.append(b.LIB) or b.LIB)
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "none.so"))
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    with pytest.raises(RuntimeError, match=r"g\+\+"):
        b.build_all()
    assert made == [b.LIB]


def test_the_binding_notices_another_torch(monkeypatch, nothing_runs, tmp_path):
    so, stamp = tmp_path / "_layer.so", tmp_path / "stamp"
    so.write_bytes(b"")
    monkeypatch.setattr(b, "BINDING", str(so))
    monkeypatch.setattr(b, "STAMP", str(stamp))
    assert not b.binding_up_to_date()  # built with what is not known
    stamp.write_text(b._host())
    assert b.binding_up_to_date() and b.build_binding() == str(so)
    stamp.write_text(b._host() + "x")
    assert not b.binding_up_to_date()
    stamp.write_text(b._host())
    os.utime(so, (1, 1))  # older than its source
    assert not b.binding_up_to_date()
