"""The bounds-checked build (libmimo_attn_checked.so, -DMIMO_CHECKED) runs the calls on
a paged cache clean: no kernel of them forms a row index outside its buffer.  The
checked library is loaded in a process of its own (MIMO_ATTN_CHECKED=1)."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_paged_calls_run_clean_under_the_checked_build():
    lib = os.path.join(ROOT, "global_attention_swa_b200", "libmimo_attn_checked.so")
    assert os.path.exists(lib), "checked build missing: run __graft_entry__.build()"
    env = dict(os.environ, MIMO_ATTN_CHECKED="1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "checked_paged_calls.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "checked ok" in r.stdout, (r.stdout[-4000:] + r.stderr[-4000:])
