"""Host side of the training operators without a GPU: offsets of dropout calls
under recomputation, and the build where parts of it are missing or changed."""
import os

import pytest
import torch
from torch.utils.checkpoint import checkpoint


@pytest.mark.parametrize("reentrant", [True, False])
def test_counter_refuses_to_move_in_a_recomputed_forward_pass(reentrant):
    from newton_schulz_05_gb300.layers import RandomCounter
    rng = RandomCounter(3)

    def inside(x):
        rng.take(x.numel())
        return (x * x).sin()

    x = torch.randn(16, requires_grad=True)
    y = checkpoint(inside, x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="recompute"):
        y.sum().backward()
    assert rng.offset == 2
    # the offset taken outside and passed in is the way
    seen = []

    def outside(x, at):
        seen.append(at)
        return (x * x).sin()

    checkpoint(outside, x, rng.take(x.numel()), use_reentrant=reentrant).sum().backward()
    assert seen == [2, 2] and rng.take(8) == 4


class Fake:
    """Stands in for build.subprocess: every command succeeds and leaves its
    output file."""

    def __init__(self):
        self.commands = []

    def run(self, cmd, **kw):
        self.commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"x")
        return type("Done", (), dict(returncode=0, stderr="", stdout=""))()


@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    from newton_schulz_05_gb300 import build
    fake = Fake()
    monkeypatch.setattr(build, "subprocess", fake)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmuon.so"))
    return build, fake


def test_library_is_built_where_the_binding_cannot_be(fake_build, monkeypatch, capsys):
    build, fake = fake_build

    def missing():
        raise build.Unavailable("no PyTorch here")

    monkeypatch.setattr(build, "_compile_binding", missing)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "no PyTorch here" in capsys.readouterr().err


def test_library_is_linked_before_a_broken_binding_is_reported(fake_build, monkeypatch):
    build, fake = fake_build

    def broken():
        raise RuntimeError("compiling the binding failed")

    monkeypatch.setattr(build, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB)


def test_missing_parts_of_pytorch_are_told_apart_from_errors(fake_build, monkeypatch):
    build, fake = fake_build
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else "/bin/true")
    with pytest.raises(build.Unavailable, match="g\\+\\+"):
        build._compile_binding()


def test_binding_is_rebuilt_for_another_pytorch(fake_build, monkeypatch):
    build, fake = fake_build
    build.build()
    first = build.binding_path()
    assert os.path.exists(first)
    n = len(fake.commands)
    build.build()
    assert len(fake.commands) == n                   # nothing to do
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    assert build.binding_path() != first and not os.path.exists(build.binding_path())
    build.build()
    assert os.path.exists(build.binding_path()) and len(fake.commands) > n


def test_a_binding_for_another_pytorch_is_not_loaded(monkeypatch):
    from newton_schulz_05_gb300 import build, layers
    build.build()
    monkeypatch.setattr(layers, "_bound", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    with pytest.raises(RuntimeError, match="not built"):
        layers._b()
