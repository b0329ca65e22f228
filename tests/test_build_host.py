"""The build where parts of the machine are missing: the C library needs nvcc alone.
A library of one small source stands in for the whole one."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from dflash_block_draft_gb300 import build as dbuild


@pytest.fixture
def small(monkeypatch, tmp_path):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (csrc / "binding.cpp").write_text("#error it does not compile\n")
    lib = tmp_path / "lib"
    lib.mkdir()
    for name, value in dict(CSRC=str(csrc), SOURCES=["one.cu"], OBJ_DIR=str(tmp_path / "obj"), LIB_DIR=str(lib),
                            LIB_PATH=str(lib / "libone.so"), BINDING_PATH=str(lib / "binding.so")).items():
        monkeypatch.setattr(dbuild, name, value)
    (lib / "binding.so").write_text("of an older build")
    return dbuild


@pytest.mark.parametrize("missing", ["torch", "headers", "compiler"])
def test_the_library_builds_without_what_only_the_binding_needs(small, monkeypatch, capsys, tmp_path, missing):
    if missing == "torch":
        monkeypatch.setattr(small.importlib.util, "find_spec", lambda name: None)
    elif missing == "headers":
        monkeypatch.setattr(small.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    assert not small.up_to_date() and small.build() == small.LIB_PATH
    assert ctypes.CDLL(small.LIB_PATH).one() == 1
    assert not os.path.exists(small.BINDING_PATH)  # the old one belongs to another library
    assert "without the Python binding" in capsys.readouterr().err
    assert small.up_to_date()


def test_a_binding_that_does_not_compile_is_an_error_after_the_library(small):
    with pytest.raises(RuntimeError, match="binding.cpp"):
        small.build()
    assert ctypes.CDLL(small.LIB_PATH).one() == 1
    assert not os.path.exists(small.BINDING_PATH) and not small.up_to_date()


def test_a_binding_for_another_torch_is_stale(small, monkeypatch, tmp_path):
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(small, "_torch_dir", lambda: str(torch))
    monkeypatch.setattr(small, "_compile_binding", lambda: "binding.o")
    run = small._run
    monkeypatch.setattr(small, "_run", lambda cmd, what: (open(cmd[cmd.index("-o") + 1], "w").close()
                                                          if what == "link of the binding" else run(cmd, what)))
    assert not small.up_to_date()
    small.build()
    assert small.up_to_date()
    (torch / "version.py").write_text("__version__ = '2'\n")
    assert not small.up_to_date()
    small.build()
    assert small.up_to_date()


@pytest.mark.parametrize("name,copied,want", [
    ("libdflash_attn.so", True, "one library"),
    ("libdflash_attn.so", False, "not built"),
    ("other.so", True, "belongs to"),
])
def test_a_library_from_another_place_brings_its_own_binding(tmp_path, name, copied, want):
    """load_library(path): the serving operators run in that library, not in a second one with an error word of
    its own."""
    pytest.importorskip("torch")
    dbuild.build()
    shutil.copy(dbuild.LIB_PATH, tmp_path / name)
    if copied:
        shutil.copy(dbuild.BINDING_PATH, tmp_path)
    code = f"""
import dflash_block_draft_gb300 as dfl
dfl.load_library({str(tmp_path / name)!r})
try:
    dfl._binding()
    maps = {{line.split()[-1] for line in open("/proc/self/maps") if "libdflash_attn" in line}}
    print("one library" if maps == {{{str(tmp_path / name)!r}}} else maps)
except RuntimeError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=dbuild.ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and want in r.stdout, (r.stdout, r.stderr[-2000:])
