"""The Python binding over a library that lacks the 8-bit key/value cache."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

PROGRAM = """
import sys
import kv_host
kv_host.build(sys.argv[1])
m = kv_host.build_binding(sys.argv[1])
try:
    m.Cache8(RuntimeError, 4096, 0, True, 2, 64).check()
except ImportError as e:
    print("refused:", e)
"""


def test_no_8_bit_cache_is_made_without_its_entry_points(tmp_path):
    """In a process of its own: a call through an entry point that is not there would end it, and the library would be found
    in the place of another test's of the same name."""
    pytest.importorskip("torch")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(tmp_path)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("refused:"), (r.returncode, r.stderr[-2000:])
