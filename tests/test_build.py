"""The build's own rules (CPU, with stand-ins for the compilers): the C library
needs no torch, and the binding's module is built again for another torch."""

import os
import subprocess
import sys
import types

import pytest
import torch

import __graft_entry__
import gqa_attention_kv_decode_gb300 as package
from gqa_attention_kv_decode_gb300 import binding, build

# writes its output file, and a line about it to $COMPILER_LOG
COMPILER = """#!/bin/sh
out=; last=
for a in "$@"; do [ "$last" = "-o" ] && out=$a; last=$a; done
case "$*" in *torch_call.cpp*) [ -n "$FAIL_CALL" ] && exit 1;; esac
echo "$out" >> "$COMPILER_LOG"
: > "$out"
"""

SCRIPT = """
import os, sys
if sys.argv[1] == "no-torch":
    sys.modules["torch"] = None  # (import torch raises ImportError)
sys.path.insert(0, {root!r})
from gqa_attention_kv_decode_gb300 import build
build.BUILD = os.path.join({tmp!r}, "_build")
build.LIB = os.path.join({tmp!r}, "libgqa_attn.so")
build.CALL = os.path.join({tmp!r}, os.path.basename(build.CALL))
assert not build.up_to_date()
print(build.build())
print(build.up_to_date())
build.build()
"""


@pytest.fixture
def tree(tmp_path):
    bin_ = tmp_path / "bin"
    bin_.mkdir()
    for name in ("nvcc", "g++"):
        (bin_ / name).write_text(COMPILER)
        (bin_ / name).chmod(0o755)
    env = dict(os.environ, PATH=f"{bin_}:{os.environ['PATH']}", NVCC=str(bin_ / "nvcc"),
               COMPILER_LOG=str(tmp_path / "log"))
    (tmp_path / "log").write_text("")

    def run(kind, **more):
        src = SCRIPT.format(root=build.ROOT, tmp=str(tmp_path))
        p = subprocess.run([sys.executable, "-c", src, kind], env=env | more, capture_output=True, text=True, timeout=300)
        made = [os.path.basename(line) for line in (tmp_path / "log").read_text().split()]
        return p, made
    return types.SimpleNamespace(run=run, path=tmp_path)


def test_the_library_is_built_without_torch(tree):
    p, made = tree.run("no-torch")
    assert p.returncode == 0, p.stderr
    assert p.stdout.split() == [str(tree.path / "libgqa_attn.so"), "True"]
    assert (tree.path / "libgqa_attn.so").exists()
    assert not any("torch_call" in m for m in made) and "no torch" in p.stderr
    assert len(made) == len(set(made))  # and once


def test_with_torch_the_module_is_built_beside_it(tree):
    p, made = tree.run("torch")
    assert p.returncode == 0, p.stderr
    assert "torch_call.o" in made and os.path.basename(build.CALL) + ".tmp" in made
    assert (tree.path / os.path.basename(build.CALL)).exists() and p.stdout.split()[1] == "True"
    assert len(made) == len(set(made))


def test_a_module_that_does_not_compile_leaves_the_library(tree):
    p, _ = tree.run("torch", FAIL_CALL="1")
    assert p.returncode != 0 and "torch_call.cpp" in p.stderr
    assert (tree.path / "libgqa_attn.so").exists()


def test_another_torch_makes_the_module_stale(monkeypatch):
    __graft_entry__.build()
    assert build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.up_to_date()


def test_the_module_is_named_for_its_python():
    assert os.path.basename(build.CALL).startswith("_torch_call.") and "3" in os.path.basename(build.CALL)
    assert os.path.basename(build.CALL) != "_torch_call.so"


@pytest.mark.parametrize("version,text", [("0.0.1", "was built for torch 0.0.1"), (None, "missing")])
def test_a_module_of_another_torch_is_not_used(monkeypatch, version, text):
    __graft_entry__.build()
    fake = None if version is None else types.SimpleNamespace(torch_version=version)
    name = package.__name__ + "._torch_call"
    monkeypatch.setitem(sys.modules, name, fake)
    if hasattr(package, "_torch_call"):
        monkeypatch.delattr(package, "_torch_call")
    if fake is not None:
        monkeypatch.setattr(package, "_torch_call", fake, raising=False)
    monkeypatch.setattr(binding, "_call_mod", None)
    with pytest.raises(RuntimeError, match=text):
        binding._call()
    monkeypatch.undo()
    assert binding._call().torch_version == torch.__version__
