"""What the build needs: the C library hipcc alone, the Python module torch and
the host's compiler too.  Nothing is compiled here."""
import sys

import pytest

from hadamard_rank_linear_amd import build as b


@pytest.fixture
def dry(monkeypatch, tmp_path):
    """build() with commands that only make their output files; their outputs."""
    made = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        if dry_fails and cmd[0] == b.CXX:
            raise RuntimeError("no compiler")
        open(out, "w").close()
        made.append(out)

    dry_fails = []
    monkeypatch.setattr(b, "_run", run)
    for name in ("OBJ", "LIB", "EXT"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    run.fails, run.made, run.path = dry_fails, made, tmp_path
    return run


def test_builds_both(dry):
    assert b.build() == b.LIB
    assert (dry.path / "LIB").exists() and (dry.path / "EXT").exists()


def test_library_without_torch(dry, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)     # as if it were not installed
    assert b.build() == b.LIB
    assert (dry.path / "LIB").exists() and not (dry.path / "EXT").exists()
    assert "_hlq_torch" in capsys.readouterr().err


def test_library_without_a_host_compiler(dry):
    dry.fails.append(True)
    with pytest.raises(RuntimeError):
        b.build()
    assert (dry.path / "LIB").exists() and not (dry.path / "EXT").exists()
