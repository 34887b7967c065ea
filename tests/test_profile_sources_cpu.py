"""The kernels' profiles in text form name the sources that they were taken on, as those are now."""
import hashlib
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_decode_attention_02_gb300", "csrc")


@pytest.mark.parametrize("profile,sources", [("quantised_cache_kernels.txt", {"sda_paged.cuh", "sda_paged.cu", "sda_quant.cuh", "sda_quant.cu"}),
                                             ("serving_step_kernels.txt", {"sda_paged.cuh", "sda_paged.cu", "sda_rope.cu", "sda_plan.cu"})])
def test_profiles_are_of_the_sources_as_they_are(profile, sources):
    with open(os.path.join(ROOT, "profiles", profile)) as f:
        named = dict(re.findall(r"^  (\w+\.cuh?) ([0-9a-f]{16})$", f.read(), re.M))
    assert set(named) == sources
    for name, digits in named.items():
        with open(os.path.join(CSRC, name), "rb") as f:
            assert hashlib.sha256(f.read()).hexdigest().startswith(digits), f"{name} has changed: {profile} is to be taken again"
