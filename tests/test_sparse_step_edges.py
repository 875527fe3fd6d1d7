"""The sparse decode step's entry points at their edges, as far as that shows
without a GPU."""
import os
import re

import pytest
import torch

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


@pytest.mark.parametrize("heads", [1, 8, 128])
def test_a_selection_workspace_holds_every_shorter_step(heads):
    """Sizes up to the 48 MiB of scores and past them, in tokens, in length and
    in heads; never more than all the step's scores, nor than the bound."""
    size = pa.pa_select_blocks_workspace_size
    tokens = [1, 2, 5, 64, 127, 128, 512, 513, 2047, 32767, 32768, 32769, 100000]
    lengths = [1, 16, 17, 100, 4096, 65536, 99999, 100000, 128000, 131072, 1 << 20, 1 << 27]
    table = [[size(T, heads, L) for L in lengths] for T in tokens]
    for i, row in enumerate(table):
        assert row == sorted(row), (tokens[i], row)
        for L, n in zip(lengths, row):
            one = size(1, heads, L)
            assert one <= n <= min(tokens[i] * one, max(48 << 20, one))
            assert n <= size(tokens[i], heads + 1, L)
    for column in zip(*table):
        assert list(column) == sorted(column)


@pytest.mark.parametrize("dtype,name", [("bfloat16", "f32"), ("uint8", "bf16"),
                                        ("uint8", "f16"), ("float16", "e4m3"),
                                        ("float32", "bf16")])
def test_a_cache_is_not_read_as_elements_of_another_size(dtype, name):
    """A type named for the cache that its elements do not have the size of: the
    kernels would read past its end, or half of it."""
    cache = torch.zeros(4, 2, 16, 128, dtype=getattr(torch, dtype))
    q = torch.zeros(1, 8, 128, dtype=torch.float32 if name == "f32" else torch.float16)
    kv = torch.zeros(1, 2, 128, dtype=q.dtype)
    i32 = dict(dtype=torch.int32)
    m = (torch.zeros(1, 4, **i32), torch.ones(1, **i32), torch.tensor([0, 1], **i32))
    slot = torch.zeros(1, dtype=torch.int64)
    sel, cnt = torch.zeros(1, 2, 1, **i32), torch.ones(1, 2, **i32)
    bounds = torch.zeros(4, 2, pa.bounds_bytes(128), dtype=torch.uint8)
    calls = [
        lambda **k: pa.pa_attention_selected(q, cache, cache.clone(), *m, 1, 1, 0.1, sel, cnt,
                                             **k),
        lambda **k: pa.pa_summarise_blocks(cache, bounds, *m, 1, 1, 1, **k),
        lambda **k: pa.pa_norm_rope_and_cache(q, kv, kv, cache, cache.clone(), slot, **k),
        lambda **k: pa.pa_attention(q, cache, cache.clone(), *m, 1, 1, 0.1, **k),
        lambda **k: pa.pa_reshape_and_cache(kv, kv, cache, cache.clone(), slot, **k),
        lambda **k: pa.pa_copy_blocks(cache, cache.clone(), torch.zeros(1, 2, dtype=torch.int64),
                                      **k)]
    for call in calls:
        with pytest.raises(ValueError, match=f"no {name} elements"):
            call(cache_dtype=name)


def test_a_stream_does_not_make_host_tensors_pass():
    """Tensors in the wrong place are named as such on a given stream too."""
    i32 = dict(dtype=torch.int32)
    q, cache = torch.zeros(1, 8, 128), torch.zeros(4, 2, 16, 128)
    m = (torch.zeros(1, 4, **i32), torch.ones(1, **i32), torch.tensor([0, 1], **i32))
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_attention_selected(q, cache, cache.clone(), *m, 1, 1, 0.1,
                                 torch.zeros(1, 2, 1, **i32), torch.ones(1, 2, **i32),
                                 workspace=ws, stream=7)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_build_step(torch.ones(1, **i32), torch.zeros(1, **i32), torch.zeros(1, 4, **i32),
                         torch.zeros(3, **i32), torch.ones(1, **i32), 8, 1, stream=7)
