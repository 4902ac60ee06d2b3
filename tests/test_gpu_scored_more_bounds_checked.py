"""The scored attention's tests of NaN, far keys, many items and edges under device-side bounds checks, as
test_gpu_scored_bounds_checked.py runs the others."""
import os
import re
import subprocess
import sys

import pytest

from test_gpu_bounds_checked import ROOT, _checked_library

pytestmark = pytest.mark.gpu


def test_more_scored_cases_pass_with_bounds_checks():
    files = ["test_gpu_scored_%s.py" % n for n in ("nan", "far", "many_items", "edges")]
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
         *[os.path.join("tests", f) for f in files]],
        cwd=ROOT, env=dict(os.environ, MHA_LIBRARY=_checked_library()), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert int(re.search(r"(\d+) passed", r.stdout).group(1)) >= 90, r.stdout[-2000:]
