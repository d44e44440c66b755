"""Linear attention, rotation, blocks and pages under the bounds-checked build."""
import os
import re

import pytest

from test_gpu_debug_bounds import _child, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu

FILES = ["test_gpu_lin.py", "test_gpu_lin_paths.py", "test_gpu_qk_norm_rope.py", "test_gpu_blocks.py",
         "test_gpu_lin_serving.py"]


def test_lin_rope_and_blocks_under_the_checked_build(debug_lib):  # noqa: F811
    files = [os.path.join("tests", f) for f in FILES]
    r = _child(["-m", "pytest", *files, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], timeout=1200)
    tail = r.stdout[-4000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert "BoundsError" not in r.stdout, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 250 and " skipped" not in r.stdout, tail
