"""Refusals of the sparse decode step's entry points, without a GPU: every
argument is checked on the host before anything is launched, so host memory
stands in for the buffers (nothing reads it)."""
import ctypes

import pytest
import torch

import paged_kv_cache_82_gb300 as pa

BUF = ctypes.create_string_buffer(1 << 22)
BASE = (ctypes.addressof(BUF) + 4095) // 4096 * 4096


def at(k):
    """The k-th 128 KiB of the buffer."""
    return BASE + k * (1 << 17)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_82_gb300 import _build
    _build.build()
    return pa.load_library()


def call(lib, name, args, **change):
    assert set(change) <= set(args), change
    return getattr(lib, name)(*{**args, **change}.values())


BUILD = dict(query_lens=at(0), computed_lens=at(1), num_seqs=4, block_tables=at(2),
             max_blocks=8, free_blocks=at(3), free_capacity=16, free_count=at(4),
             free_count_out=at(5), num_blocks=64, block_size=16, num_tokens=32,
             seq_lens=at(6), qsl=at(7), positions=at(8), slots=at(9), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(num_seqs=-1), 1), (dict(num_tokens=-1), 1), (dict(max_blocks=-1), 1),
    (dict(free_capacity=-1), 1), (dict(num_blocks=0), 1), (dict(block_size=32), 2),
    (dict(num_seqs=16385), 2), (dict(num_tokens=1 << 31), 2), (dict(max_blocks=1 << 27), 2),
    (dict(query_lens=None), 1), (dict(computed_lens=None), 1), (dict(block_tables=None), 1),
    (dict(free_blocks=None), 1), (dict(free_count=None), 1), (dict(free_count_out=None), 1),
    (dict(seq_lens=None), 1), (dict(qsl=None), 1), (dict(positions=None), 1),
    (dict(slots=None), 1), (dict(slots=at(9) + 4), 1), (dict(qsl=at(7) + 2), 1),
    (dict(seq_lens=at(0)), 1), (dict(positions=at(9) + 8), 1), (dict(block_tables=at(3)), 1),
    (dict(seq_lens=at(1) + 4), 1), (dict(free_count_out=at(6)), 1),
])
def test_build_step_refuses(lib, change, status):
    assert call(lib, "pa_build_step", BUILD, **change) == status


ROPE = dict(q=at(0), k=at(1), v=at(2), dtype=pa.PA_BF16, num_tokens=4, q_stride=1024,
            k_stride=256, v_stride=256, q_weight=at(3), k_weight=at(4),
            weight_dtype=pa.PA_BF16, eps=1e-6, cos_sin=at(5), max_position=64,
            rotary_dim=128, interleaved=0, positions=at(6), q_out=at(7), k_cache=at(8),
            v_cache=at(10), cache_dtype=pa.PA_BF16, num_blocks=4, block_size=16,
            num_q_heads=8, num_kv_heads=2, head_dim=128, slots=at(12), k_scale=1.0,
            v_scale=1.0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=pa.PA_FP8_E4M3), 2), (dict(dtype=9), 1), (dict(cache_dtype=pa.PA_F16), 2),
    (dict(head_dim=96), 2), (dict(block_size=8), 2), (dict(num_kv_heads=0), 1),
    (dict(num_q_heads=0), 1), (dict(num_tokens=-1), 1), (dict(q_stride=1023), 1),
    (dict(k_stride=255), 1), (dict(v_stride=255), 1), (dict(rotary_dim=24), 2),
    (dict(rotary_dim=144), 2), (dict(rotary_dim=-16), 1), (dict(weight_dtype=pa.PA_F16), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(q_out=None), 1), (dict(k_cache=None), 1), (dict(slots=None), 1),
    (dict(cos_sin=None), 1), (dict(positions=None), 1), (dict(cos_sin=at(5) + 4), 1),
    (dict(q_out=at(7) + 8), 1), (dict(k_cache=at(8) + 8), 1), (dict(q=at(0) + 1), 1),
    (dict(k_cache=at(10)), 1), (dict(q_out=at(1)), 1), (dict(q_out=at(8)), 1),
    (dict(q_out=at(0), q_stride=1032), 1), (dict(max_position=-1), 1),
    (dict(cache_dtype=pa.PA_FP8_E4M3, k_scale=0.0), 1),
    (dict(cache_dtype=pa.PA_NVFP4, v_scale=float("inf")), 1),
])
def test_norm_rope_and_cache_refuses(lib, change, status):
    assert call(lib, "pa_norm_rope_and_cache", ROPE, **change) == status


STEP = dict(block_tables=at(2), max_blocks=8, seq_lens=at(3), qsl=at(4), num_seqs=2,
            num_tokens=2, max_query_len=1, max_seq_len=128)
BAD_STEP = [
    (dict(num_seqs=-1), 1), (dict(num_tokens=-1), 1), (dict(max_query_len=-1), 1),
    (dict(max_seq_len=-1), 1), (dict(max_seq_len=129), 1), (dict(block_tables=None), 1),
    (dict(seq_lens=None), 1), (dict(qsl=None), 1), (dict(qsl=at(4) + 2), 1),
    (dict(block_size=8), 2), (dict(head_dim=80), 2), (dict(num_kv_heads=0), 1),
    (dict(num_blocks=0), 1)]

SUM = dict(k_cache=at(0), cache_dtype=pa.PA_BF16, num_blocks=8, block_size=16,
           num_kv_heads=2, head_dim=128, **STEP, bounds=at(6), stream=None)


@pytest.mark.parametrize("change,status", BAD_STEP + [
    (dict(cache_dtype=7), 1), (dict(k_cache=None), 1), (dict(bounds=None), 1),
    (dict(bounds=at(6) + 8), 1), (dict(bounds=at(0)), 1), (dict(bounds=at(3)), 1)])
def test_summarise_blocks_refuses(lib, change, status):
    assert call(lib, "pa_summarise_blocks", SUM, **change) == status


SELECT = dict(q=at(0), q_dtype=pa.PA_BF16, bounds=at(1), num_blocks=8, block_size=16,
              num_q_heads=8, num_kv_heads=2, head_dim=128, **STEP, max_selected=4,
              keep_first=1, keep_last=1, selected=at(5), num_selected=at(6),
              workspace=at(7), workspace_bytes=1 << 17, stream=None)


@pytest.mark.parametrize("change,status", BAD_STEP + [
    (dict(q_dtype=pa.PA_INT4), 2), (dict(num_q_heads=7), 1), (dict(max_selected=0), 1),
    (dict(keep_first=-1), 1), (dict(keep_last=0), 1), (dict(keep_first=4), 1),
    (dict(keep_first=2 ** 31 - 1, keep_last=2 ** 31 - 1), 1), (dict(q=None), 1),
    (dict(bounds=None), 1), (dict(selected=None), 1), (dict(num_selected=None), 1),
    (dict(workspace=None), 1), (dict(workspace_bytes=127), 1), (dict(workspace=at(7) + 16), 1),
    (dict(selected=at(0)), 1), (dict(num_selected=at(5)), 1), (dict(workspace=at(1)), 1),
    (dict(q=at(0) + 8), 1)])
def test_select_blocks_refuses(lib, change, status):
    assert call(lib, "pa_select_blocks", SELECT, **change) == status


ATTEND = dict(q=at(0), q_dtype=pa.PA_BF16, k_cache=at(8), v_cache=at(10),
              cache_dtype=pa.PA_BF16, num_blocks=8, block_size=16, num_q_heads=8,
              num_kv_heads=2, head_dim=128, **STEP, selected=at(5), num_selected=at(6),
              max_selected=4, scale=0.1, k_scale=1.0, v_scale=1.0, out=at(7),
              workspace=at(12), workspace_bytes=1 << 17, stream=None)


@pytest.mark.parametrize("change,status", BAD_STEP + [
    (dict(q_dtype=pa.PA_NVFP4), 2), (dict(cache_dtype=pa.PA_F16), 2),
    (dict(q_dtype=pa.PA_F32, cache_dtype=pa.PA_FP8_E4M3), 2), (dict(num_q_heads=9), 1),
    (dict(max_selected=0), 1), (dict(scale=float("inf")), 1),
    (dict(cache_dtype=pa.PA_FP8_E4M3, k_scale=-1.0), 1), (dict(q=None), 1),
    (dict(k_cache=None), 1), (dict(selected=None), 1), (dict(num_selected=None), 1),
    (dict(out=None), 1), (dict(k_cache=at(8) + 64), 1), (dict(out=at(7) + 8), 1)])
def test_attention_selected_refuses(lib, change, status):
    assert call(lib, "pa_attention_selected", ATTEND, **change) == status


def test_attention_selected_limits(lib):
    """Sizes whose counts the kernels hold in 31 bits are refused beyond them."""
    assert call(lib, "pa_attention_selected", ATTEND, max_selected=(1 << 24) + 1) == 2
    assert call(lib, "pa_attention_selected", ATTEND, num_tokens=1 << 30) == 2


def test_nothing_to_do_is_no_error(lib):
    """No requests, tokens or keys: PA_OK, and no buffer is looked at."""
    none = dict.fromkeys(("block_tables", "seq_lens", "qsl"))
    assert call(lib, "pa_summarise_blocks", SUM, num_seqs=0, **none) == 0
    assert call(lib, "pa_select_blocks", SELECT, num_tokens=0, q=None, **none) == 0
    assert call(lib, "pa_attention_selected", ATTEND, max_query_len=0, out=None, **none) == 0
    assert call(lib, "pa_norm_rope_and_cache", ROPE, num_tokens=0, q=None, k=None) == 0


def test_select_workspace_size():
    """Scores of as many tokens as 48 MiB hold, of one token at least."""
    size = pa.pa_select_blocks_workspace_size
    assert size(0, 8, 131072) == 0
    assert size(1, 8, 131072) == 8192 * 8 * 4
    assert size(64, 8, 16) == 64 * 8 * 4 * 4        # one block, rows of four
    assert size(100000, 8, 131072) == (48 << 20)
    assert size(4, 64, (1 << 31) - 16) == 4 * 64 * ((1 << 27) - 1 + 1)
    with pytest.raises(pa.PaError):
        size(-1, 8, 16)


def _cpu(**kw):
    i32 = dict(dtype=torch.int32)
    a = dict(q=torch.zeros(2, 8, 128, dtype=torch.bfloat16),
             k_cache=torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16),
             block_tables=torch.zeros(2, 4, **i32), seq_lens=torch.ones(2, **i32),
             query_start_loc=torch.tensor([0, 1, 2], **i32),
             bounds=torch.zeros(4, 2, pa.bounds_bytes(128), dtype=torch.uint8))
    a.update(kw)
    return a


def test_binding_refuses_tensors_the_abi_would_misread():
    """Shapes, types, layouts and places are checked before a pointer is taken
    (CPU tensors: the last check)."""
    def select(**kw):
        a = _cpu(**kw)
        return pa.pa_select_blocks(a["q"], a["bounds"], a["block_tables"], a["seq_lens"],
                                   a["query_start_loc"], 1, 1, 2,
                                   workspace=torch.empty(64, dtype=torch.uint8))

    def attend(sel=(2, 2, 3), **kw):
        a = _cpu(**kw)
        return pa.pa_attention_selected(
            a["q"], a["k_cache"], a["k_cache"].clone(), a["block_tables"], a["seq_lens"],
            a["query_start_loc"], 1, 1, 0.1, torch.zeros(*sel, dtype=torch.int32),
            torch.zeros(2, 2, dtype=torch.int32), workspace=torch.empty(64, dtype=torch.uint8))

    def rope(**kw):
        t = dict(q=torch.zeros(2, 8, 128), key=torch.zeros(2, 2, 128),
                 value=torch.zeros(2, 2, 128), k_cache=torch.zeros(4, 2, 16, 128),
                 v_cache=torch.zeros(4, 2, 16, 128),
                 slot_mapping=torch.zeros(2, dtype=torch.int64))
        t.update(kw)
        return pa.pa_norm_rope_and_cache(**t)

    for f, kw, what in [
            (select, {}, "CUDA"), (attend, {}, "CUDA"), (rope, {}, "CUDA"),
            (select, dict(bounds=torch.zeros(4, 2, 100, dtype=torch.uint8)), "bounds"),
            (select, dict(q=torch.zeros(2, 16, 128)[:, ::2]), "contiguous"),
            (select, dict(seq_lens=torch.ones(2, dtype=torch.int64)), "seq_lens"),
            (attend, dict(sel=(2, 3, 3)), "selected"),
            (attend, dict(query_start_loc=torch.zeros(2, dtype=torch.int32)), "sequences"),
            (rope, dict(key=torch.zeros(2, 2, 128, dtype=torch.float16)), "one type"),
            (rope, dict(q=torch.zeros(2, 128, 8).transpose(1, 2)), "contiguous"),
            (rope, dict(cos_sin=torch.zeros(4, 128)), "positions"),
            (rope, dict(cos_sin=torch.zeros(4, 128), positions=torch.zeros(2)), "positions"),
            (rope, dict(slot_mapping=torch.zeros(2, dtype=torch.int32)), "slot_mapping"),
            (rope, dict(q_weight=torch.zeros(64)), "q_weight"),
            (rope, dict(q_weight=torch.zeros(128), k_weight=torch.zeros(128).half()), "k_weight"),
            (rope, dict(q_out=torch.zeros(2, 8, 64)), "q_out")]:
        with pytest.raises(ValueError, match=what):
            f(**kw)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="query_lens"):
        pa.pa_build_step(torch.zeros(2), torch.zeros(2, **i32), torch.zeros(2, 4, **i32),
                         torch.zeros(3, **i32), torch.zeros(1, **i32), 8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_build_step(torch.zeros(2, **i32), torch.zeros(2, **i32),
                         torch.zeros(2, 4, **i32), torch.zeros(3, **i32),
                         torch.zeros(1, **i32), 8, 4)
