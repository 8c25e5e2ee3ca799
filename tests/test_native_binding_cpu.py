"""The native part of the binding: left out where it was not built, an error where it is
there and does not load.  CPU only."""

import os
import subprocess
import sys
import sysconfig

import pytest

import global_attention_swa_b200 as mimo

NAME = "_fast_call" + sysconfig.get_config_var("EXT_SUFFIX")


@pytest.mark.parametrize("broken", [False, True])
def test_a_native_part_that_does_not_load_is_an_error(tmp_path, broken):
    package = tmp_path / "global_attention_swa_b200"
    package.mkdir()
    home = os.path.dirname(os.path.abspath(mimo.__file__))
    for name in os.listdir(home):
        if not name.startswith(("_fast_call", "__pycache__")):
            os.symlink(os.path.join(home, name), package / name)
    if broken:
        (package / NAME).write_bytes(b"no shared object")
    r = subprocess.run([sys.executable, "-c", "import global_attention_swa_b200 as m; print('native:', m._fast)"],
                       cwd=tmp_path, env=dict(os.environ, PYTHONPATH=str(tmp_path)), capture_output=True, text=True, timeout=300)
    if broken:
        assert r.returncode != 0 and "ImportError" in r.stderr and "_fast_call" in r.stderr
    else:
        assert r.returncode == 0 and "native: None" in r.stdout, r.stderr
