"""What build() compiles again."""
import pytest

from moe_expert_offload_router_gb300 import build as b


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """build() with its compilers replaced by notes, after a build that is up to date."""
    b.build()
    done = []
    made = tmp_path / "made_for.txt"
    made.write_text(open(b.MADE_FOR).read())
    monkeypatch.setattr(b, "MADE_FOR", str(made))
    monkeypatch.setattr(b, "_compile", lambda src, verbose: done.append("kernel"))
    monkeypatch.setattr(b, "_link", lambda objs: done.append("library"))
    monkeypatch.setattr(b, "_compile_binding", lambda: done.append("binding"))
    monkeypatch.setattr(b, "_link_binding", lambda obj: done.append("module"))
    return done, made


def test_nothing_is_compiled_twice(steps):
    b.build()
    assert steps[0] == []


@pytest.mark.parametrize("other", ["2.0.0", ""])
def test_a_binding_for_another_torch_is_compiled_again(steps, monkeypatch, other):
    done, made = steps
    made.write_text(made.read_text().replace(made.read_text().splitlines()[-2], other))
    b.build()
    assert done == ["binding", "module"]   # the library does not depend on torch
    b.build()
    assert len(done) == 2


def test_a_binding_for_another_python_is_compiled_again(steps, monkeypatch):
    done, made = steps
    monkeypatch.setattr(b.sys, "version", "3.99.0 (another)")
    b.build()
    assert done == ["binding", "module"]


def test_a_binding_that_says_nothing_is_compiled_again(steps):
    done, made = steps
    made.unlink()
    b.build()
    assert done == ["binding", "module"]


def test_force_compiles_all(steps):
    b.build(force=True)
    assert steps[0].count("kernel") == len(b.sources()) and {"library", "binding", "module"} <= set(steps[0])
