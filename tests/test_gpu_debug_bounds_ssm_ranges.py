"""The state space prefill's range, segment and workspace tests, the maps'
errors and the norm's halves under the bounds-checked build."""
import os
import re

import pytest

from test_gpu_debug_bounds import _child, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu

FILES = ["test_gpu_ssm_ranges.py", "test_gpu_ssm_segments.py", "test_ssm_workspace.py", "test_ssm_refusals.py",
         "test_gpu_batch_maps_errors.py", "test_gpu_add_rmsnorm_ties.py"]


def test_ranges_and_segments_under_the_checked_build(debug_lib):  # noqa: F811
    files = [os.path.join("tests", f) for f in FILES]
    r = _child(["-m", "pytest", *files, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], timeout=1200)
    tail = r.stdout[-4000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert "BoundsError" not in r.stdout, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 100 and " skipped" not in r.stdout, tail
