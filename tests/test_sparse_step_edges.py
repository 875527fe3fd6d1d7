"""The sparse decode step's entry points at their edges, as far as that shows
without a GPU."""
import os
import re

import paged_kv_cache_82_gb300 as pa

CSRC = os.path.join(os.path.dirname(os.path.abspath(pa.__file__)), "csrc")


def _kernel(text, name):
    """The body of the kernel of this name."""
    begin = text.index("{", text.index(f" {name}("))
    depth = 0
    for i in range(begin, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[begin:i]
    raise AssertionError(name)


def test_words_that_a_step_replaces_are_not_read_as_constants():
    """pa_build_step updates lengths, block tables and the stack's height in
    place: a load that needs memory nobody writes (__ldg) may be made again
    behind the write, so none of these is read by one."""
    with open(os.path.join(CSRC, "step_kernels.cu")) as f:
        body = _kernel(f.read(), "build_step_kernel")
    constant = set(re.findall(r"__ldg\(\s*&?p\.(\w+)", body))
    assert "free_blocks" in constant  # never written
    in_place = {"computed_lens", "free_count", "block_tables"}
    assert all(f"p.{w}" in body for w in in_place) and not in_place & constant
