"""The scored attention's and the shared-prefix decoding's tests under device-side bounds checks: the build of
test_gpu_bounds_checked.py, in which every TMA coordinate and direct global store is checked against the problem's
extents and a failed check records MHA_ERR_BOUNDS in the status word, which those tests assert to be zero."""
import os
import re
import subprocess
import sys

import pytest

from test_gpu_bounds_checked import ROOT, _checked_library

pytestmark = pytest.mark.gpu


def test_scored_cases_pass_with_bounds_checks():
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
         os.path.join("tests", "test_gpu_scored.py"), os.path.join("tests", "test_gpu_decode_shared.py"),
         "-k", "not largest_length"],
        cwd=ROOT, env=dict(os.environ, MHA_LIBRARY=_checked_library()), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert int(re.search(r"(\d+) passed", r.stdout).group(1)) >= 140, r.stdout[-2000:]
