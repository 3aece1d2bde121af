"""The scored, rotary and page calls in the debug-checks build: every index they form is checked before
its use."""
import os
import subprocess
import sys

import pytest

from test_gpu_debug_build import ROOT, _debug_lib

pytestmark = pytest.mark.gpu


@pytest.mark.timeout(900)
def test_more_paged_calls_pass_every_check():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_debug_paged_more_cases.py")],
                       env=dict(os.environ, YOCO_LIB_PATH=_debug_lib()), capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug cases ok" in r.stdout
