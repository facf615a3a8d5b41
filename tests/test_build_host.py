"""The build: which extension module a process loads, and processes that build at once.  No GPU."""

import os
import stat
import subprocess
import sys

import pytest

from rotated_bit_kv_kvq_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# stands for nvcc and for the C++ compiler: notes the call, writes its output in two halves with a pause between
FAKE = """#!/usr/bin/env python3
import os, sys, time
out = sys.argv[sys.argv.index("-o") + 1]
with open(os.environ["FAKE_LOG"], "a") as f:
    f.write(os.path.basename(out) + "\\n")
with open(out, "w") as f:
    f.write("first half, ")
    f.flush()
    time.sleep(0.3)
    f.write("second half")
"""

CHILD = """
import os, sys, time
from rotated_bit_kv_kvq_gb300 import build as b
b.BUILD = sys.argv[1]
b.LIB = os.path.join(b.BUILD, "libkvq.so")
time.sleep(max(0.0, float(sys.argv[2]) - time.time()))
print(open(b.ensure_built()).read())
print(open(b.ensure_binding()).read())
"""


def test_processes_that_build_at_once_build_once(tmp_path):
    import time
    pytest.importorskip("torch")
    fake = tmp_path / "compiler"
    fake.write_text(FAKE)
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    log, out = tmp_path / "log", tmp_path / "build"
    env = dict(os.environ, NVCC=str(fake), CXX=str(fake), FAKE_LOG=str(log), PYTHONPATH=ROOT)
    start = str(time.time() + 3.0)
    procs = [subprocess.Popen([sys.executable, "-c", CHILD, str(out), start], env=env, cwd=ROOT, stdout=subprocess.PIPE,
                              stderr=subprocess.PIPE, text=True) for _ in range(4)]
    for p in procs:
        got, err = p.communicate(timeout=120)
        assert p.returncode == 0, err
        assert got.splitlines() == ["first half, second half"] * 2
    calls = log.read_text().splitlines()
    assert len(calls) == len(set(calls)) == len(build._sources()) + 2


def test_the_binding_belongs_to_one_torch_and_one_python(monkeypatch):
    torch = pytest.importorskip("torch")
    import sysconfig
    here = build.binding_path()
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "99.0.1+cu999")
    assert build.binding_path() != here
    monkeypatch.undo()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: ".cpython-399-x.so" if n == "EXT_SUFFIX" else real(n))
    assert build.binding_path() != here
