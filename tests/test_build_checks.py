"""Building the binding's native argument checks where that cannot be done (no
GPU needed)."""
import subprocess

import pytest

from combine_ep_get_dispatch_amd import build as B


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, ["g++"])])
def test_a_failed_build_leaves_none(tmp_path, monkeypatch, capsys, error):
    """No compiler, or one that fails: the build goes on, and no file of an
    earlier one is loaded."""
    out = tmp_path / "_checks.so"
    out.write_bytes(b"of an earlier build")

    def run(cmd, **kw):
        (tmp_path / "_checks.so.tmp").write_bytes(b"half of it")
        raise error

    monkeypatch.setattr(B.subprocess, "run", run)
    assert B.build_checks(str(out)) is None
    assert not list(tmp_path.iterdir())
    assert "not built" in capsys.readouterr().err
