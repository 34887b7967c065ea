"""The quantised cache's kernels are launched before their predecessor is done, too: each waits before it touches memory."""
import re

import pytest

from test_dependent_launch_cpu import body


@pytest.mark.parametrize("name,kernel", [("sda_quant.cu", "sda_quantised_append_kernel"), ("sda_quant.cu", "sda_quantised_read_kernel"),
                                         ("sda_paged.cu", "sda_region_extent_kernel")])
def test_memory_is_touched_after_the_wait(name, kernel):
    text = body(name, kernel)
    ahead = text[text.index("{"):text.index("pdl_wait()")]
    assert not re.search(r"p\.\w+\[|\*p\.|slot_of\(|atomic", ahead)
    assert "p." in text[text.index("pdl_wait()"):]
