"""The state space, residual norm and batch map tests under the bounds-checked
build: every index those cases reach stays in its buffer's bounds.  Left out:
the tensors beyond 32 bits, whose indices are checked against their results."""
import os
import re

import pytest

from test_gpu_debug_bounds import _child, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu

FILES = ["test_gpu_ssm.py", "test_gpu_ssm_paths.py", "test_gpu_ssm_decode_paths.py", "test_gpu_add_rmsnorm.py",
         "test_gpu_batch_maps.py", "test_gpu_serving_step.py"]


def test_state_space_norm_and_maps_under_the_checked_build(debug_lib):  # noqa: F811
    files = [os.path.join("tests", f) for f in FILES]
    r = _child(["-m", "pytest", *files, "-m", "gpu", "-k", "not beyond_32_bits", "-x", "-q", "-p",
                "no:cacheprovider"], timeout=1200)
    tail = r.stdout[-4000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert "BoundsError" not in r.stdout, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 200 and " skipped" not in r.stdout, tail
