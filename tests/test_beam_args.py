"""Refusals of beam selection, forked and compacted rows, copies and moves of all
layers, without a GPU: every argument is checked on the host before anything is
launched, so host memory stands in for the buffers (nothing reads it)."""
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


BEAM = dict(logits=at(0), dtype=pa.PA_F32, groups=2, width=4, vocab=1000, stride=1024,
            beam_scores=at(1), finished=at(2), end_token=2, num_selected=4, scores=at(3),
            parents=at(4), tokens=at(5), finished_out=at(6), workspace=at(7),
            workspace_bytes=1 << 17, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=9), 1), (dict(dtype=pa.PA_FP8_E4M3), 2), (dict(dtype=pa.PA_INT4), 2),
    (dict(groups=-1), 1), (dict(width=0), 1), (dict(width=65), 2), (dict(vocab=0), 1),
    (dict(vocab=(1 << 24) + 1, stride=1 << 25), 2), (dict(stride=999), 1),
    (dict(num_selected=0), 1), (dict(num_selected=129), 2), (dict(groups=1 << 22), 2),
    (dict(end_token=-2), 1), (dict(end_token=1000), 1), (dict(end_token=-1), 1),
    (dict(logits=None), 1), (dict(beam_scores=None), 1), (dict(scores=None), 1),
    (dict(parents=None), 1), (dict(tokens=None), 1), (dict(workspace=None), 1),
    (dict(workspace=at(7) + 16), 1), (dict(workspace_bytes=255), 1),
    (dict(logits=at(0) + 2), 1), (dict(scores=at(3) + 2), 1), (dict(tokens=at(5) + 1), 1),
    (dict(scores=at(4)), 1), (dict(parents=at(0)), 1), (dict(tokens=at(7)), 1),
    (dict(scores=at(1), num_selected=3), 1), (dict(scores=at(1) + 4), 1),
    (dict(finished_out=at(2), num_selected=8), 1), (dict(finished_out=at(1)), 1)])
def test_beam_select_refuses(lib, change, status):
    assert call(lib, "pa_beam_select", BEAM, **change) == status


ROWS = dict(tables=at(1), tables_out=at(2), max_blocks=8, seq_lens=at(3), lens_out=at(4),
            refs=at(5), refs_out=at(6), num_blocks=64, block_size=16, free_blocks=at(7),
            capacity=64, free_count=at(8), free_count_out=at(9))
BAD_ROWS = [
    (dict(rows=-1), 1), (dict(rows=4097), 2), (dict(max_blocks=-1), 1),
    (dict(max_blocks=1 << 27), 2), (dict(rows=4096, max_blocks=1 << 18), 2),
    (dict(num_blocks=0), 1), (dict(num_blocks=1 << 31), 2), (dict(block_size=8), 2),
    (dict(capacity=-1), 1), (dict(capacity=1 << 31), 2), (dict(tables=None), 1),
    (dict(tables_out=None), 1), (dict(seq_lens=None), 1), (dict(lens_out=None), 1),
    (dict(refs=None), 1), (dict(refs_out=None), 1), (dict(free_blocks=None), 1),
    (dict(free_count=None), 1), (dict(free_count_out=None), 1), (dict(workspace=None), 1),
    (dict(workspace=at(12) + 64), 1), (dict(workspace_bytes=31), 1), (dict(tables=at(1) + 2), 1),
    (dict(refs_out=at(6) + 1), 1), (dict(tables_out=at(1) + 4), 1), (dict(lens_out=at(1)), 1),
    (dict(refs_out=at(5) + 4), 1), (dict(refs_out=at(7)), 1), (dict(free_count_out=at(2)), 1),
    (dict(workspace=at(5)), 1), (dict(free_count=at(7)), 1)]
FORK = dict(sources=at(0), rows=4, **ROWS, mapping=at(10), num_pairs=at(11), workspace=at(12),
            workspace_bytes=1 << 17, stream=None)


@pytest.mark.parametrize("change,status", BAD_ROWS + [
    (dict(sources=None), 1), (dict(sources=at(0) + 2), 1), (dict(mapping=None), 1),
    (dict(mapping=at(10) + 4), 1), (dict(num_pairs=None), 1), (dict(mapping=at(0)), 1),
    (dict(num_pairs=at(9)), 1), (dict(lens_out=at(0)), 1)])
def test_fork_blocks_refuses(lib, change, status):
    assert call(lib, "pa_fork_blocks", FORK, **change) == status


COMPACT = dict(keep=at(0), max_keep=40, keep_lens=at(13), keep_start=at(14), rows=4, **ROWS,
               src=at(10), dst=at(11), moves=at(15), workspace=at(12), workspace_bytes=1 << 17,
               stream=None)


@pytest.mark.parametrize("change,status", BAD_ROWS + [
    (dict(max_keep=-1), 1), (dict(max_keep=1 << 29), 2), (dict(max_keep=2 ** 31 - 1, rows=1), 2),
    (dict(keep=None), 1), (dict(keep_lens=None), 1), (dict(src=None), 1), (dict(dst=None), 1),
    (dict(moves=None), 1), (dict(src=at(10) + 4), 1), (dict(moves=at(15) + 2), 1),
    (dict(keep_start=at(14) + 1), 1), (dict(src=at(11)), 1), (dict(dst=at(0)), 1),
    (dict(moves=at(13)), 1), (dict(lens_out=at(14)), 1)])
def test_compact_blocks_refuses(lib, change, status):
    assert call(lib, "pa_compact_blocks", COMPACT, **change) == status


# a layer: 8 blocks of 2 heads of 16 x 128 bf16 = 64 KiB
LAYERS = dict(k=at(0), v=at(4), dtype=pa.PA_BF16, layers=3, k_stride=1 << 17, v_stride=1 << 17,
              num_blocks=8, block_size=16, heads=2, head_dim=128)
BAD_LAYERS = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=at(0) + 8), 1), (dict(dtype=6), 1),
    (dict(layers=0), 1), (dict(layers=(1 << 16) + 1), 2), (dict(k_stride=(1 << 16) - 16), 1),
    (dict(v_stride=(1 << 17) + 8), 1), (dict(k_stride=-(1 << 17)), 1), (dict(num_blocks=0), 1),
    (dict(block_size=32), 2), (dict(heads=0), 1), (dict(head_dim=96), 2), (dict(v=at(0)), 1),
    (dict(v=at(1)), 1), (dict(v=at(0) + (1 << 15)), 1), (dict(v=at(2), v_stride=1 << 16), 1)]
COPY = dict(**LAYERS, mapping=at(8), max_pairs=5, num_pairs=at(9), stream=None)


@pytest.mark.parametrize("change,status", BAD_LAYERS + [
    (dict(mapping=None), 1), (dict(mapping=at(8) + 4), 1), (dict(max_pairs=-1), 1),
    (dict(max_pairs=1 << 31), 2), (dict(num_pairs=at(9) + 2), 1), (dict(mapping=at(1)), 1),
    (dict(num_pairs=at(4) + 64), 1)])
def test_copy_blocks_layers_refuses(lib, change, status):
    assert call(lib, "pa_copy_blocks_layers", COPY, **change) == status


MOVE = dict(**LAYERS, src=at(8), dst=at(9), moves=at(10), rows=4, max_moves=20, stream=None)


@pytest.mark.parametrize("change,status", BAD_LAYERS + [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(moves=None), 1), (dict(src=at(8) + 4), 1),
    (dict(moves=at(10) + 2), 1), (dict(rows=-1), 1), (dict(max_moves=-1), 1),
    (dict(max_moves=1 << 30), 2), (dict(rows=1 << 27), 2), (dict(dst=at(0)), 1),
    (dict(moves=at(6)), 1)])
def test_move_tokens_refuses(lib, change, status):
    assert call(lib, "pa_move_tokens", MOVE, **change) == status


def test_nothing_to_do_is_no_error(lib):
    assert call(lib, "pa_beam_select", BEAM, groups=0, logits=None, workspace=None) == 0
    assert call(lib, "pa_copy_blocks_layers", COPY, max_pairs=0, mapping=None) == 0
    assert call(lib, "pa_move_tokens", MOVE, rows=0, src=None) == 0
    assert call(lib, "pa_move_tokens", MOVE, max_moves=0, dst=None) == 0


def test_workspace_sizes():
    """Room for what the kernels write, none of it dependent on the device."""
    # one chunk of 2048 logits per row: 8 keys of 8 bytes, padded, and a pair
    assert pa.pa_beam_select_workspace_size(1, 1, 2041, 8) == 256 + 8
    assert pa.pa_beam_select_workspace_size(1, 1, 2042, 8) == 256 + 16
    assert pa.pa_beam_select_workspace_size(0, 4, 1000, 8) == 0
    # rows enough for chunks of 8192
    assert pa.pa_beam_select_workspace_size(100, 4, 8185, 4) == 400 * 4 * 8 + 400 * 8
    assert pa.pa_fork_blocks_workspace_size(0, 7) == 0
    assert pa.pa_fork_blocks_workspace_size(5, 257) == 4 * (5 + 5 * 2)
    assert pa.pa_compact_blocks_workspace_size(5, 257) >= 4 * 5 * 257
    for f, bad in ((pa.pa_beam_select_workspace_size, (1, 65, 100, 1)),
                   (pa.pa_beam_select_workspace_size, (-1, 1, 100, 1)),
                   (pa.pa_fork_blocks_workspace_size, (-1, 3)),
                   (pa.pa_compact_blocks_workspace_size, (3, -1))):
        with pytest.raises(pa.PaError):
            f(*bad)


def test_workspace_of_the_largest_step_serves_smaller_ones():
    """The size never falls as groups, beams, tokens or picks grow: the kernels' plan
    changes from short chunks to long ones on the way."""
    size = pa.pa_beam_select_workspace_size
    for V in (1, 2041, 2042, 8185, 8186, 32000, 100_000, 128_256, 1 << 24):
        for K in (1, 8, 128):
            rows = [size(g, 1, V, K) for g in range(0, 70)]
            assert rows == sorted(rows)
            assert [size(1, w, V, K) for w in range(1, 65)] == rows[1:65]
    for g in (1, 2, 3, 5, 15, 16, 40):
        of_tokens = [size(g, 1, V, 4) for V in range(1, 140_000, 997)]
        assert of_tokens == sorted(of_tokens)
    rows = [pa.pa_fork_blocks_workspace_size(r, 300) for r in range(60)]
    assert rows == sorted(rows)
    rows = [pa.pa_compact_blocks_workspace_size(7, m) for m in range(0, 3000, 31)]
    assert rows == sorted(rows)


def test_binding_refuses_tensors_the_abi_would_misread():
    """Shapes, types, layouts and places are checked before a pointer is used (CPU
    tensors: the last check)."""
    i32 = dict(dtype=torch.int32)

    def beam(logits=torch.zeros(8, 100), scores=torch.zeros(2, 4), **kw):
        return pa.pa_beam_select(logits, scores, 4, **kw)

    def rows(**kw):
        a = dict(block_tables=torch.zeros(3, 5, **i32), seq_lens=torch.zeros(3, **i32),
                 extra_refs=torch.zeros(9, **i32), free_blocks=torch.zeros(9, **i32),
                 free_count=torch.zeros(1, **i32))
        a.update(kw)
        return a

    def fork(sources=torch.zeros(3, **i32), **kw):
        return pa.pa_fork_blocks(sources, **rows(**kw))

    def compact(keep=torch.zeros(3, 4, **i32), keep_lens=torch.zeros(3, **i32), **kw):
        return pa.pa_compact_blocks(keep, keep_lens, **rows(**kw))

    def copy(k=torch.zeros(2, 4, 2, 16, 64), v=None, m=torch.zeros(3, 2, dtype=torch.int64), **kw):
        return pa.pa_copy_blocks_layers(k, torch.zeros_like(k) if v is None else v, m, **kw)

    def move(src=torch.zeros(3, 2, dtype=torch.int64), dst=None, **kw):
        k = torch.zeros(2, 4, 2, 16, 64)
        return pa.pa_move_tokens(k, k.clone(), src, src.clone() if dst is None else dst,
                                 torch.zeros(3, **i32), **kw)

    for f, kw, what in [
            (beam, {}, "CUDA"), (fork, {}, "CUDA"), (compact, {}, "CUDA"), (copy, {}, "CUDA"),
            (move, {}, "CUDA"),
            (beam, dict(logits=torch.zeros(7, 100)), "beam_scores"),
            (beam, dict(logits=torch.zeros(100, 8).t()), "contiguous rows"),
            (beam, dict(logits=torch.zeros(1, 100).expand(8, 100)), "overlap"),
            (beam, dict(scores=torch.zeros(2, 4, dtype=torch.float64)), "beam_scores"),
            (beam, dict(finished=torch.zeros(2, 4)), "finished"),
            (beam, dict(finished=torch.zeros(2, 3, dtype=torch.uint8)), "finished"),
            (beam, dict(tokens=torch.zeros(2, 4, dtype=torch.int64)), "tokens"),
            (beam, dict(parents=torch.zeros(2, 5, **i32)), "parents"),
            (fork, dict(sources=torch.zeros(3, dtype=torch.int64)), "sources"),
            (fork, dict(sources=torch.zeros(4, **i32)), "sources"),
            (fork, dict(block_tables=torch.zeros(15, **i32)), "block_tables"),
            (fork, dict(block_tables_out=torch.zeros(5, 3, **i32)), "block_tables_out"),
            (fork, dict(block_tables=torch.zeros(5, 3, **i32).t()), "block_tables"),
            (fork, dict(extra_refs_out=torch.zeros(8, **i32)), "extra_refs_out"),
            (fork, dict(free_count=torch.zeros(2, **i32)), "free_count"),
            (fork, dict(num_pairs=torch.zeros(1)), "num_pairs"),
            (compact, dict(keep=torch.zeros(3, **i32)), "keep"),
            (compact, dict(keep=torch.zeros(2, 4, **i32)), "keep"),
            (compact, dict(keep_start=torch.zeros(3)), "keep_start"),
            (compact, dict(src_slots=torch.zeros(3, 4, dtype=torch.int64)), "src_slots"),
            (copy, dict(k=torch.zeros(4, 2, 16)), "caches"),
            (copy, dict(v=torch.zeros(2, 4, 2, 16, 64).half()), "alike"),
            (copy, dict(k=torch.zeros(2, 4, 2, 64, 16).transpose(3, 4)), "contiguous"),
            (copy, dict(m=torch.zeros(6, dtype=torch.int64)), "block_mapping"),
            (copy, dict(k=torch.zeros(0, 4, 2, 16, 64)), "layer"),
            (copy, dict(cache_dtype="e4m3"), "elements"),
            (copy, dict(k=torch.zeros(4, 2, 100, dtype=torch.uint8), cache_dtype="int4"),
             "page size"),
            (move, dict(src=torch.zeros(6, dtype=torch.int64)), "src_slots"),
            (move, dict(dst=torch.zeros(3, 3, dtype=torch.int64)), "src_slots")]:
        with pytest.raises(ValueError, match=what):
            f(**kw)
