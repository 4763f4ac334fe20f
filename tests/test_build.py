"""The library needs nvcc alone; torch and Python's headers are the binding's."""
import os
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "paged_kv_decode_16_gb300", "build.py")

NVCC = """#!/bin/sh
# writes its output and a line of its log
echo "$@" >> {log}
while [ "$1" != -o ]; do shift; done
: > "$2"
"""

RUN = """
import importlib.util, os, sys
sys.modules.update({blocked})
spec = importlib.util.spec_from_file_location("pkv_build", {build!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.OUT_DIR = {out!r}
b.LIB = os.path.join(b.OUT_DIR, "libpagedkv.so")
{body}
"""


@pytest.fixture
def run(tmp_path):
    """run(body, blocked modules) -> (its process, the lines of nvcc's calls)."""
    log = tmp_path / "log"
    nvcc = tmp_path / "cuda" / "bin" / "nvcc"
    nvcc.parent.mkdir(parents=True)
    nvcc.write_text(NVCC.format(log=log))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)

    def go(body, blocked="dict(torch=None)"):
        log.write_text("")
        r = subprocess.run([sys.executable, "-c", RUN.format(
            blocked=blocked, build=BUILD, out=str(tmp_path / "out"), body=body)],
            capture_output=True, text=True, env=dict(os.environ, CUDA_HOME=str(tmp_path / "cuda")))
        return r, log.read_text().splitlines()
    go.lib = tmp_path / "out" / "libpagedkv.so"
    return go


def test_library_without_torch(run):
    r, calls = run("print(b.build_library())")
    assert r.returncode == 0 and r.stdout.split() == [str(run.lib)], r.stderr
    assert run.lib.exists() and sum("-shared" in c for c in calls) == 1
    r, calls = run("print(b.build_library())")  # nothing is newer
    assert r.returncode == 0 and calls == []


def test_command_without_torch(run):
    """What a user of the C library runs: the library, and no word about an error."""
    r, calls = run("b.main([])")
    assert r.returncode == 0 and str(run.lib) in r.stdout, r.stderr
    assert run.lib.exists() and calls


def test_binding_that_does_not_compile_leaves_the_library(run):
    body = """
import subprocess
b._compile_binding = lambda out: subprocess.CompletedProcess([], 1, "", "no Python.h")
b.binding_path = lambda: os.path.join(b.OUT_DIR, "calls.so")
try:
    b.build()
except RuntimeError as e:
    print("raised", e)
"""
    r, calls = run(body, "{}")
    assert r.returncode == 0 and "no Python.h" in r.stdout, r.stderr
    assert run.lib.exists()


def test_another_torch_compiles_the_binding_alone(run):
    body = """
import subprocess
def compiled(out):
    print("binding")
    return subprocess.CompletedProcess([], 0, "", "")
b._compile_binding = compiled
b._link_binding = lambda obj: open(b.binding_path(), "w").close()
b.binding_path = lambda: os.path.join(b.OUT_DIR, NAME)
b.build()
"""
    r, calls = run("NAME = 'one.so'\n" + body, "{}")
    assert r.returncode == 0 and r.stdout.split() == ["binding"] and calls, r.stderr
    r, calls = run("NAME = 'one.so'\n" + body, "{}")
    assert r.returncode == 0 and r.stdout.split() == [] and calls == [], r.stderr
    r, calls = run("NAME = 'two.so'\n" + body, "{}")
    assert r.returncode == 0 and r.stdout.split() == ["binding"] and calls == [], r.stderr
