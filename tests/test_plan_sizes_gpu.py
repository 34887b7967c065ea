"""Request counts around the kernel's shared memory limits, in a process that has made no larger
call before: what one call raises stays raised for those after it."""
import os
import random
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# 24 bytes a request beside under 1 KB of the kernel's own: 48 KB without a raised limit
SIZES = [1, 1999, 2005, 2015, 2016, 2047, 2048, 2049, 4096, 8192]


def first_calls():
    import test_plan_gpu
    for n in SIZES:
        r = random.Random(n)
        test_plan_gpu.check(*test_plan_gpu.problem(r, n, 16, 90, 0, 5, spare=3), in_place=bool(n & 1))


def test_each_size_before_any_larger():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", "import test_plan_sizes_gpu as t; t.first_calls()"], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
