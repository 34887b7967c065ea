"""Kernels that are launched before their predecessor is done: each waits before it touches memory,
and one that reads inputs ahead of its wait follows a kernel that has waited by then."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_decode_attention_02_gb300", "csrc")


def body(name, kernel):
    """The source of a kernel, from its name to the closing brace of its function."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    at = re.search(rf"__global__[^;{{]*\b{kernel}\(", text).start()
    return text[at:text.index("\n}\n", at)]


def test_the_split_kernel_waits_before_it_lets_the_combine_kernel_start():
    split, combine = body("sdattn.cu", "sda_split_kernel"), body("sdattn.cu", "sda_combine_kernel")
    assert combine.index("p.gate[") < combine.index("pdl_wait()")              # it reads the gate ahead of its wait,
    assert split.index("pdl_wait()") < split.index("pdl_launch_dependents()")  # so this order is needed


def test_the_serving_step_kernels_touch_memory_after_their_wait():
    for name, kernel in (("sda_plan.cu", "sda_plan_kernel"), ("sda_rope.cu", "sda_rope_kernel"),
                         ("sda_paged.cuh", "sda_paged_kernel"), ("sda_paged.cu", "sda_paged_join_kernel")):
        text = body(name, kernel)
        ahead = text[text.index("{"):text.index("pdl_wait()")]
        assert not re.search(r"p\.\w+\[|\*p\.", ahead), kernel
