"""What build() compiles and when, with the compilers replaced by records of
their calls."""
import json
import os
import subprocess

import pytest


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """The build module on files of its own; calls: the outputs it has compiled."""
    from block_sparse_long_05_b200 import build
    calls = []

    def compiler(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        calls.append(os.path.basename(out).split(".")[0])
        with open(out, "w") as f:
            f.write("built")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_msa_torch.so"))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "_msa_torch.json"))
    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    return build, calls


def test_binding_is_built_once(fake):
    build, calls = fake
    assert build.build_binding() == build.BINDING
    assert build.build_binding() == build.BINDING
    assert calls == ["_msa_torch"]


@pytest.mark.parametrize("name, value", [("torch", "1.0"), ("cxx11_abi", None), ("python", "cpython-30")])
def test_binding_of_another_torch_or_python_is_built_anew(fake, name, value):
    build, calls = fake
    build.build_binding()
    with open(build.BINDING_KEY) as f:
        key = json.load(f)
    assert name in key
    key[name] = value
    with open(build.BINDING_KEY, "w") as f:
        json.dump(key, f)
    build.build_binding()
    build.build_binding()
    assert calls == ["_msa_torch"] * 2


@pytest.mark.parametrize("record", [None, "", "{"])
def test_binding_without_a_record_is_built_anew(fake, record):
    build, calls = fake
    build.build_binding()
    if record is None:
        os.remove(build.BINDING_KEY)
    else:
        with open(build.BINDING_KEY, "w") as f:
            f.write(record)
    build.build_binding()
    assert calls == ["_msa_torch"] * 2


def test_failed_binding_leaves_no_record(fake, monkeypatch):
    """A module whose compilation failed is not taken for a current one."""
    build, calls = fake

    def broken(cmd, **_):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build.subprocess, "check_call", broken)
    with pytest.raises(subprocess.CalledProcessError):
        build.build_binding()
    assert not os.path.exists(build.BINDING) and not os.path.exists(build.BINDING_KEY)


def test_library_does_not_need_the_binding(fake, monkeypatch):
    """Without a C++ compiler the library is built all the same, and build() says
    what is missing."""
    build, calls = fake
    order = []
    monkeypatch.setattr(build, "build_library", lambda *a, **k: order.append("library"))

    def missing(cmd, **_):
        order.append("binding")
        raise FileNotFoundError(cmd[0])

    monkeypatch.setattr(build.subprocess, "check_call", missing)
    with pytest.raises(FileNotFoundError):
        build.build()
    assert order == ["library", "binding"]
