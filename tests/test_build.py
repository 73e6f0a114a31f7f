"""build.py's handling of files, with a stand-in for the compiler."""

import concurrent.futures
import os
import stat
import sys

import pytest

from matrix_optimizers_sharded_amd import build as b

COMPILER = """#!{python}
import os, sys, time
out = sys.argv[sys.argv.index("-o") + 1]
inputs = [a for a in sys.argv[1:] if a.endswith((".hip", ".o")) and a != out]
time.sleep(float(os.environ["COMPILER_SECONDS"]))
if os.environ.get("COMPILER_FAILS") == os.path.basename(inputs[0]):
    sys.exit("no")
if "-c" in sys.argv:
    text = [a for a in sys.argv if a.startswith("-cuid")] + [os.path.basename(inputs[0])]
else:
    text = [open(i).read() for i in inputs]
open(out, "w").write(" ".join(text) + "\\n")
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    cc = tmp_path / "cc"
    cc.write_text(COMPILER.format(python=sys.executable))
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(b, "HIPCC", str(cc))
    monkeypatch.setattr(b, "PKG", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib" / "libmatopt.so"))
    monkeypatch.setenv("COMPILER_SECONDS", "0.05")
    return tmp_path


def test_builds_at_once_do_not_disturb_each_other(place):
    with concurrent.futures.ThreadPoolExecutor(max_workers=6) as pool:
        libs = list(pool.map(lambda _: b.build(), range(6)))
    assert set(libs) == {b.LIB}
    text = open(b.LIB).read()
    for src in b.SOURCES:
        assert os.path.basename(src) in text
    assert os.listdir(place / "lib") == ["libmatopt.so"]          # nothing left behind


def test_a_failed_build_keeps_the_library_that_was_there(place, monkeypatch):
    b.build()
    before = open(b.LIB).read()
    monkeypatch.setenv("COMPILER_FAILS", os.path.basename(b.SOURCES[0]))
    with pytest.raises(RuntimeError):
        b.build()
    assert open(b.LIB).read() == before
    assert os.listdir(place / "lib") == ["libmatopt.so"]


def test_the_units_names_in_the_code_do_not_come_from_their_place(place):
    """The compiler makes a unit's id from its paths unless it is given one."""
    b.build()
    for src in b.SOURCES:
        assert f"-cuid={os.path.splitext(os.path.basename(src))[0]} " in open(b.LIB).read()
