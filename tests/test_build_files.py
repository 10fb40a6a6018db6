"""What a build leaves behind, and that nothing built is in the repository."""
import os
import subprocess

import pytest

from causal_depthwise_conv1d_gb300 import build

ROOT = build.ROOT


def test_no_built_binary_is_tracked():
    if not os.path.isdir(os.path.join(ROOT, ".git")):
        pytest.skip("not a git checkout")
    names = subprocess.run(["git", "ls-files", "-z"], cwd=ROOT, check=True, stdout=subprocess.PIPE).stdout
    for name in names.decode().split("\0")[:-1]:
        path = os.path.join(ROOT, name)
        if os.path.isfile(path):
            with open(path, "rb") as f:
                assert f.read(4) != b"\x7fELF", name


@pytest.mark.parametrize("fails", ["compilation", "link"])
def test_a_failed_build_leaves_no_file(fails, tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "a.cpp").write_text("#error no\n" if fails == "compilation" else "int x;\n")
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "ext.so"))
    monkeypatch.setattr(build, "_ext_command", lambda out: ["sh", "-c", f"echo > '{out}'"])

    def no_link(*args, **kw):
        raise subprocess.CalledProcessError(1, args[0])

    monkeypatch.setattr(build.subprocess, "run", no_link)
    with pytest.raises((RuntimeError, subprocess.CalledProcessError)):
        build.build(force=True)
    assert sorted(os.listdir(tmp_path)) == ["_build", "csrc"]
    assert all(n.endswith(".o") for n in os.listdir(tmp_path / "_build"))
