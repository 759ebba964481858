"""The build: the C library needs no torch, and the binding is made anew for another torch."""
import os
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Builds into a folder of its own with compilers that only write their output files.
SCRIPT = """
import os, sys
sys.path.insert(0, {root!r})
if {hide}:
    sys.modules["torch"] = None              # importing it raises ImportError
import multistage_smem_pipeline_gb300.build as b
b.OBJ_DIR, b.LIB_DIR = {out!r} + "/obj", {out!r} + "/lib"
b.LIB, b.BINDING = b.LIB_DIR + "/libgemm_tn_f16.so", b.LIB_DIR + "/_experts.so"
b.nvcc = lambda: {bin!r} + "/nvcc"
b.build()
print("library", os.path.exists(b.LIB), "binding", os.path.exists(b.BINDING), "again", not b.up_to_date())
"""


@pytest.fixture
def compilers(tmp_path):
    folder = tmp_path / "bin"
    folder.mkdir()
    for name in ("nvcc", "g++"):
        exe = folder / name
        exe.write_text("#!/bin/sh\n"
                       f"echo {name} \"$@\" >> {tmp_path}/calls\n"
                       f"[ -e {tmp_path}/fail_{name} ] && exit 1\n"
                       "while [ $# -gt 0 ]; do [ \"$1\" = -o ] && : > \"$2\"; shift; done\n")
        exe.chmod(exe.stat().st_mode | stat.S_IXUSR)
    return tmp_path


def run(compilers, hide=False):
    script = SCRIPT.format(root=ROOT, out=str(compilers), bin=str(compilers / "bin"), hide=hide)
    env = dict(os.environ, PATH=f"{compilers / 'bin'}:{os.environ['PATH']}")
    return subprocess.run([sys.executable, "-c", script], env=env, text=True, capture_output=True)


def test_the_library_is_built_without_torch(compilers):
    """A machine that has nvcc alone gets the C library."""
    done = run(compilers, hide=True)
    assert done.returncode == 0, done.stderr
    assert "library True binding False" in done.stdout


def test_the_library_is_built_where_the_binding_is_not(compilers):
    """A binding that does not compile is an error, and the library is there all the same."""
    (compilers / "fail_g++").touch()
    done = run(compilers)
    assert done.returncode != 0 and "experts_binding.cpp" in done.stderr
    assert (compilers / "lib" / "libgemm_tn_f16.so").exists()


def test_both_are_built(compilers):
    done = run(compilers)
    assert "library True binding True again False" in done.stdout, done.stderr


def test_the_binding_is_made_anew_for_another_torch(compilers):
    assert "again False" in run(compilers).stdout
    assert "again False" in run(compilers).stdout
    calls = (compilers / "calls").read_text().count("experts_binding.cpp -o")
    assert calls == 1                                 # the second time nothing was compiled
    stamp = compilers / "lib" / "_experts.built_for"
    made_for = stamp.read_text()
    for other in (made_for.replace("torch", "torch 0.1"), made_for + "x", ""):
        stamp.write_text(other)
        assert "again False" in run(compilers).stdout
        assert stamp.read_text() == made_for
        calls += 1
        assert (compilers / "calls").read_text().count("experts_binding.cpp -o") == calls
    stamp.unlink()
    run(compilers)
    assert stamp.read_text() == made_for


def test_the_library_is_built_where_torch_does_not_import(compilers):
    """A torch that is there and broken is an error, after the library."""
    broken = compilers / "broken" / "torch"
    broken.mkdir(parents=True)
    (broken / "__init__.py").write_text("raise ImportError('a broken torch')\n")
    script = SCRIPT.format(root=ROOT, out=str(compilers), bin=str(compilers / "bin"), hide=False)
    env = dict(os.environ, PATH=f"{compilers / 'bin'}:{os.environ['PATH']}",
               PYTHONPATH=str(compilers / "broken"))
    done = subprocess.run([sys.executable, "-c", script], env=env, text=True, capture_output=True)
    assert done.returncode != 0 and "a broken torch" in done.stderr
    assert (compilers / "lib" / "libgemm_tn_f16.so").exists()
