"""Building the module of the 8-bit calls: what it needs, when it is built
anew, and what is left where it cannot be (with compilers that only write down
how they were called)."""
import os
import stat
import sys
import warnings

import pytest
import torch

from post_weight_quantization_accumulate_b200 import build as build_mod
from post_weight_quantization_accumulate_b200 import w8a8

# writes its output file, as a compiler of before version 13: -nostdlib++ is not known
OLD_COMPILER = """#!/bin/sh
echo "$@" >> "$0.log"
for a in "$@"; do
    if [ "$a" = -nostdlib++ ]; then echo "unrecognized command-line option '-nostdlib++'" >&2; exit 1; fi
    if [ "$last" = -o ]; then echo built > "$a"; fi
    last="$a"
done
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The module's files at a place of their own; the library is the real one."""
    build_mod.build()
    monkeypatch.setattr(build_mod, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build_mod, "CALLS_STAMP", str(tmp_path / "calls.txt"), raising=False)
    for name, text in (("old", OLD_COMPILER), ("none", "#!/bin/sh\necho no torch headers >&2; exit 1\n")):
        (tmp_path / name).write_text(text)
        os.chmod(tmp_path / name, stat.S_IRWXU)

    def use(name):
        monkeypatch.setenv("CXX", str(tmp_path / name))
        monkeypatch.setenv("CC", str(tmp_path / name))
    use("old")
    return tmp_path, use


def _calls(place):
    log = place[0] / "old.log"
    return len(log.read_text().splitlines()) if log.exists() else 0


def test_compilers_before_version_13_build_it(place):
    assert build_mod.build_calls() == str(place[0] / "_calls.so")
    assert (place[0] / "_calls.so").read_text() == "built\n"


def test_it_is_built_anew_for_another_torch_only(place, monkeypatch):
    build_mod.build_calls()
    n = _calls(place)
    build_mod.build_calls()
    assert _calls(place) == n
    monkeypatch.setattr(torch, "__version__", "3.0")
    build_mod.build_calls()
    assert _calls(place) == 2 * n
    build_mod.build_calls()
    assert _calls(place) == 2 * n


def test_the_library_stands_where_the_module_cannot_be_built(place):
    """Of use to everything but w8a8: build() warns; nothing stale is left."""
    (place[0] / "_calls.so").write_text("stale")
    os.utime(place[0] / "_calls.so", (1, 1))
    place[1]("none")
    with pytest.warns(RuntimeWarning, match="no torch headers"):
        assert build_mod.build() == build_mod.LIB
    assert os.path.exists(build_mod.LIB) and not (place[0] / "_calls.so").exists()
    with pytest.raises(RuntimeError, match="no torch headers"):
        build_mod.build_calls()
    assert sorted(p.name for p in place[0].iterdir() if p.name.startswith("_calls")) == []


def test_the_library_stands_without_torch(place, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="torch"):
        assert build_mod.build() == build_mod.LIB


def test_a_built_tree_is_left_alone(place):
    build_mod.build_calls()
    place[1]("none")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert build_mod.build() == build_mod.LIB


def test_w8a8_says_what_is_missing(monkeypatch):
    build_mod.build()
    monkeypatch.setattr(w8a8, "_native", None)
    exists = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: exists(p) and not str(p).endswith("_calls.so"))
    with pytest.raises(RuntimeError, match="_calls.so is missing"):
        w8a8.quantize_tokens(torch.zeros(1, 16))
