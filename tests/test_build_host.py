"""The build without a torch, with a binding that does not compile, and with
another torch: the library needs nvcc alone, and is not made again for the
module's sake.  (The compilers are stand-ins that write their output file and a
line to a log.)"""
import importlib.metadata
import os
import sys

import pytest

from speculative_decode_verify_paged_gb300 import build as libbuild

COMPILER = """#!{python}
import sys
if {fail}:
    sys.exit("does not compile")
out = sys.argv[sys.argv.index("-o") + 1]
open(out, "w").write("made")
open({log!r}, "a").write({name!r} + "\\n")
"""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    log = tmp_path / "log"

    def make(name, fail=False):
        path = tmp_path / name
        path.write_text(COMPILER.format(python=sys.executable, fail=fail, log=str(log), name=name))
        path.chmod(0o755)
        return str(path)

    def used():
        lines = log.read_text().split() if log.exists() else []
        log.write_text("")
        return {n: lines.count(n) for n in set(lines)}

    out = tmp_path / "_build"
    monkeypatch.setattr(libbuild, "BUILD", str(out))
    monkeypatch.setattr(libbuild, "LIB", str(out / "libspec_attn.so"))
    monkeypatch.setattr(libbuild, "CALLS", str(out / "spec_attn_calls.so"))
    monkeypatch.setenv("NVCC", make("nvcc"))
    monkeypatch.setenv("CXX", make("cxx"))
    make.used = used
    return make


N = len(libbuild.sources()) + 1        # one call a source and one to link


def test_without_torch(tools, monkeypatch):
    find, version = libbuild.importlib.util.find_spec, importlib.metadata.version

    def no_version(name):
        if name == "torch":
            raise importlib.metadata.PackageNotFoundError(name)
        return version(name)
    monkeypatch.setattr(libbuild.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(libbuild.importlib.metadata, "version", no_version)
    assert libbuild.build() == libbuild.LIB
    assert os.path.exists(libbuild.LIB) and not os.path.exists(libbuild.CALLS)
    assert tools.used() == {"nvcc": N}
    libbuild.build()
    assert tools.used() == {}


def test_a_binding_that_does_not_compile_leaves_the_library(tools, monkeypatch):
    good = os.environ["CXX"]
    libbuild.build()
    assert tools.used() == {"nvcc": N, "cxx": 2} and os.path.exists(libbuild.CALLS)
    monkeypatch.setenv("CXX", tools("bad", fail=True))
    with pytest.raises(RuntimeError, match="does not compile"):
        libbuild.build(force=True)
    assert tools.used() == {"nvcc": N}
    assert os.path.exists(libbuild.LIB) and not os.path.exists(libbuild.CALLS)      # (nor an older module)
    with pytest.raises(RuntimeError, match="does not compile"):
        libbuild.build()
    assert tools.used() == {}                                                       # the library is up to date
    monkeypatch.setenv("CXX", good)
    libbuild.build()
    assert tools.used() == {"cxx": 2} and os.path.exists(libbuild.CALLS)
    libbuild.build()
    assert tools.used() == {}


def test_another_torch_makes_the_module_again(tools, monkeypatch):
    libbuild.build()
    tools.used()
    monkeypatch.setattr(libbuild.importlib.metadata, "version", lambda name: "0.0.0")
    libbuild.build()
    assert tools.used() == {"cxx": 2}
    libbuild.build()
    assert tools.used() == {}
