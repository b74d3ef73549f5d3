"""Which files a build depends on: a library older than any of them is built again."""

import os
import re

import pytest

from amsgrad_optimizer_step_gb300 import build


def test_every_included_file_is_a_dependency():
    """Whatever the sources include with quotes, directly or not, is among the dependencies."""
    deps = {os.path.realpath(d) for d in build._deps()}
    todo, seen = list(build.sources()), set()
    while todo:
        path = todo.pop()
        with open(path) as f:
            names = re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M)
        for name in names:
            found = [p for p in (os.path.join(d, name) for d in (build.CSRC, build.INCLUDE))
                     if os.path.exists(p)]
            assert found, f"{path} includes {name}"
            if found[0] not in seen:
                seen.add(found[0])
                todo.append(found[0])
    assert any(p.endswith(".cuh") for p in seen)
    missing = [p for p in seen if os.path.realpath(p) not in deps]
    assert not missing


@pytest.mark.parametrize("name", ["a.cu", "b.cpp", "c.h", "d.cuh"])
def test_a_changed_file_makes_the_library_stale(tmp_path, monkeypatch, name):
    for f in ("a.cu", "b.cpp", "c.h", "d.cuh"):
        (tmp_path / f).write_text("")
        os.utime(tmp_path / f, (1000, 1000))
    lib = tmp_path / "lib.so"
    lib.write_text("")
    this = os.path.getmtime(build.__file__)
    os.utime(lib, (this + 10, this + 10))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    monkeypatch.setattr(build, "_built_for_this_host", lambda path: True)
    assert build.up_to_date(str(lib))
    os.utime(tmp_path / name, (this + 20, this + 20))
    assert not build.up_to_date(str(lib))
