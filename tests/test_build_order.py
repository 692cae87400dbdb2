"""The library needs hipcc alone: it is linked also where the binding's tensor
checks (torch, the Python headers) cannot be compiled, which is then reported."""

import subprocess

import pytest

from bit_nf4_quantized_amd import build


def test_the_library_is_linked_without_the_tensor_checks(monkeypatch, tmp_path):
    linked = []

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("linked")
        linked.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def no_torch():
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / build.LIB_NAME))
    monkeypatch.setattr(build, "_compile", lambda src: str(tmp_path / (src + ".o")))
    monkeypatch.setattr(build, "_build_tensors", no_torch)
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(ImportError):
        build.build()
    assert len(linked) == 1 and all(str(tmp_path / (s + ".o")) in linked[0] for s in build.SOURCES)
    assert (tmp_path / build.LIB_NAME).read_text() == "linked"
