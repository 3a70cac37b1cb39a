"""The build without what only the native calls need (torch, a host compiler), with a
stand-in for hipcc that makes empty files."""
import os
import stat

import pytest

from two_sided_hessian_amd import build


@pytest.fixture
def stub(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "HIPCC", str(hipcc))
    for name, path in (("BUILD", "_build"), ("LIB", "lib.so"), ("FAST", "_fast.so")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    return tmp_path


def files(path):
    return sorted(f for f in os.listdir(path) if ".so" in f)


def no_torch(out):
    raise ImportError("no torch here")


@pytest.mark.parametrize("command", [no_torch, lambda out: ["/no/such/compiler", out],
                                     lambda out: ["sh", "-c", f": > {out}; echo no good; exit 1"]])
def test_the_library_is_built_without_the_native_calls(stub, monkeypatch, capfd, command):
    (stub / "_fast.so").write_text("another build's")
    monkeypatch.setattr(build, "fast_command", command)
    assert build.build() == build.LIB
    assert files(stub) == ["lib.so"]                              # and nothing that might not fit it
    assert "_fast.so is not built" in capfd.readouterr().err


def test_both_are_built(stub, monkeypatch, capfd):
    monkeypatch.setattr(build, "fast_command", lambda out: ["sh", "-c", f": > {out}"])
    build.build()
    assert files(stub) == ["_fast.so", "lib.so"] and not capfd.readouterr().err


def test_a_source_that_does_not_compile_fails_the_build(stub, monkeypatch):
    with open(build.HIPCC, "w") as f:
        f.write("#!/bin/sh\necho broken; exit 1\n")
    monkeypatch.setattr(build, "fast_command", lambda out: ["sh", "-c", f": > {out}"])
    with pytest.raises(RuntimeError, match="broken"):
        build.build()
    assert files(stub) == []
