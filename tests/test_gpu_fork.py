"""pa_fork_blocks and pa_compact_blocks against plain loops, exactly."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _beam_ref as ref

pytestmark = pytest.mark.gpu

FLAGS = {"metadata": pa.PA_DEV_ERR_METADATA, "blocks": pa.PA_DEV_ERR_NO_BLOCKS,
         "block id": pa.PA_DEV_ERR_BLOCK_ID}


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _tree(rng, groups, width, hi, free, spare=0):
    """Rows that share full blocks as beams do (each with those of the row before it,
    up to some block), lengths alike within a group: a dict of the calls' state."""
    R = groups * width
    lens = np.repeat(rng.integers(0, hi + 1, groups), width)
    M = max(1, -(-int(lens.max()) // 16)) + int(rng.integers(0, 3))
    table = np.full((R, M), -7, np.int64)
    n = 0
    for r in range(R):
        nb = -(-int(lens[r]) // 16)
        cut = int(rng.integers(0, lens[r] // 16 + 1)) if r % width else 0
        table[r, :cut] = table[r - 1, :cut]
        table[r, cut:nb] = np.arange(n, n + nb - cut)
        n += nb - cut
    NB = n + free + 3
    ids = rng.permutation(NB)
    used = table >= 0
    table[used] = ids[table[used]]
    extra = np.maximum(np.bincount(table[used], minlength=NB) - 1, 0)
    stack = np.full(n + free + 3 + spare, -5)
    stack[:free] = ids[n:n + free]
    return dict(table=table.astype(np.int32), lens=lens.astype(np.int32),
                refs=extra.astype(np.int32), stack=stack.astype(np.int32), count=free)


def _fork(c, sources, in_place=True, capacity=None):
    stack = c["stack"] if capacity is None else c["stack"][:capacity]
    table, lens, refs, st = (_i32(x) for x in (c["table"], c["lens"], c["refs"], stack))
    count = _i32([c["count"]])
    before = c["table"] if in_place else np.full_like(c["table"], -11)
    outs = {} if in_place else dict(
        block_tables_out=_i32(before), seq_lens_out=torch.empty_like(lens),
        extra_refs_out=torch.empty_like(refs), free_count_out=torch.empty_like(count))
    mapping, pairs = pa.pa_fork_blocks(_i32(sources), table, lens, refs, st, count, **outs)
    flags = pa.pa_get_device_error()
    want = ref.fork(np.asarray(sources), c["table"], c["lens"], c["refs"], stack, c["count"],
                    before)
    if not in_place:
        for t, k in ((table, "table"), (lens, "lens"), (refs, "refs")):
            np.testing.assert_array_equal(t.cpu().numpy(), c[k])
        assert int(count) == c["count"]
        table, lens, refs, count = (outs[k] for k in (
            "block_tables_out", "seq_lens_out", "extra_refs_out", "free_count_out"))
    for name, t in (("table", table), ("seq_lens", lens), ("refs", refs), ("stack", st),
                    ("pairs", mapping)):
        np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=name)
    assert (int(count), int(pairs)) == (want["count"], want["num_pairs"])
    assert flags == sum(FLAGS[f] for f in want["flags"])
    return want


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("sources", [
    [0, 1, 2, 3], [0, 0, 0, 0], [3, 2, 1, 0], [1, 1, 2, 2], [-1, 0, -1, 2], [-1] * 4,
    [2, -1, 2, 2]])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 48, 61])
def test_four_rows(in_place, sources, length):
    rng = np.random.default_rng(length)
    c = _tree(rng, 1, 4, 0, 0)
    nb = -(-length // 16)
    c["lens"][:] = length
    c["table"] = np.full((4, nb + 1), -3, np.int32)
    # the first block, where full, is shared by all; the rest is each row's own
    shared = 1 if length >= 16 else 0
    for r in range(4):
        own = nb - shared
        c["table"][r, :nb] = [0] * shared + list(range(1 + r * own, 1 + (r + 1) * own))
    c["refs"] = np.zeros(40, np.int32)
    c["refs"][0] = 3 if shared else 0
    c["stack"] = np.arange(30, 70, dtype=np.int32) % 40
    c["count"] = 5
    assert not _fork(c, sources, in_place)["flags"]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("groups,width,hi", [
    (1, 1, 100), (1, 3, 40), (16, 4, 700), (5, 7, 5000), (128, 8, 300), (300, 5, 90),
    (1024, 4, 40), (1, 2, 70000)])
def test_beams(in_place, groups, width, hi):
    rng = np.random.default_rng(groups + hi)
    c = _tree(rng, groups, width, hi, 9)
    src = np.sort(rng.integers(0, width, (groups, width)), 1) + np.arange(groups)[:, None] * width
    src = src.reshape(-1)
    assert not _fork(c, src, in_place)["flags"]
    # any row from any row, some ended
    src = rng.integers(-1, groups * width, groups * width)
    want = _fork(c, src, in_place)
    assert want["flags"] <= {"blocks"}


@pytest.mark.parametrize("groups,width,hi", [(8, 4, 300), (150, 8, 3000)])
def test_captured_calls_on_two_streams(groups, width, hi):
    """A graph of a fork and one of a compaction, each on buffers of its own, replayed at
    the same time: one cluster, and a grid of every SM."""
    rng = np.random.default_rng(groups)
    c = _tree(rng, groups, width, hi, 9, spare=groups * width * hi // 16)
    R = groups * width
    src = np.sort(rng.integers(0, width, (groups, width)), 1) + np.arange(groups)[:, None] * width
    d = _tree(rng, groups, 1, hi, 40, spare=groups * hi // 16)
    keep, ks, start = _lists(rng, d, 0.3)
    fork_in = [_i32(c[k]) for k in ("table", "lens", "refs", "stack")] + [_i32([c["count"]])]
    comp_in = [_i32(d[k]) for k in ("table", "lens", "refs", "stack")] + [_i32([d["count"]])]
    sources, kd, kl, st = _i32(src.reshape(-1)), _i32(keep), _i32(ks), _i32(start)

    def outs(t):
        return dict(block_tables_out=t[0].clone(), seq_lens_out=t[1].clone(),
                    extra_refs_out=t[2].clone(), free_count_out=t[4].clone())

    fo, co = outs(fork_in), outs(comp_in)
    torch.cuda.synchronize()
    graphs, got = [], []
    for which in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if which == 0:
                got.append(pa.pa_fork_blocks(sources, *fork_in, **fo))
            else:
                got.append(pa.pa_compact_blocks(kd, kl, *comp_in, keep_start=st, **co))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    want = ref.fork(src.reshape(-1), c["table"], c["lens"], c["refs"], c["stack"], c["count"])
    np.testing.assert_array_equal(fo["block_tables_out"].cpu().numpy(), want["table"])
    np.testing.assert_array_equal(fo["extra_refs_out"].cpu().numpy(), want["refs"])
    np.testing.assert_array_equal(got[0][0].cpu().numpy(), want["pairs"])
    assert int(fo["free_count_out"]) == want["count"] and R == len(want["seq_lens"])
    moves = got[1][2].cpu().numpy()
    want = ref.compact(keep, ks, start, d["table"], d["lens"], d["refs"], d["stack"], d["count"],
                       got[1][0].cpu().numpy(), got[1][1].cpu().numpy())
    np.testing.assert_array_equal(moves, want["moves"])
    np.testing.assert_array_equal(got[1][0].cpu().numpy(), want["src"])
    np.testing.assert_array_equal(got[1][1].cpu().numpy(), want["dst"])
    np.testing.assert_array_equal(co["extra_refs_out"].cpu().numpy(), want["refs"])
    assert int(co["free_count_out"]) == want["count"]


def test_a_step_of_beams_needs_no_spare_block():
    """With no free block at all, the copies go into what the step gives back."""
    rng = np.random.default_rng(3)
    for seed in range(20):
        c = _tree(np.random.default_rng(seed), 6, 5, 200, 0)
        src = rng.integers(0, 5, (6, 5)) + np.arange(6)[:, None] * 5
        assert not _fork(c, src.reshape(-1))["flags"]


def test_rows_that_part_from_one_prompt_and_the_block_held_outside():
    """A prompt's row taken over by idle rows; its last block is also held by another
    request, so that even the first row gets a copy."""
    for extra in (0, 1, 2):
        for length in (20, 32, 33):
            table = np.full((5, 6), -1, np.int32)
            nb = -(-length // 16)
            table[3, :nb] = np.arange(10, 10 + nb)
            refs = np.zeros(64, np.int32)
            refs[10 + nb - 1] = extra
            lens = np.array([0, 0, 0, length, 0], np.int32)
            c = dict(table=table, lens=lens, refs=refs, count=8,
                     stack=np.arange(40, 60, dtype=np.int32))
            want = _fork(c, [3, 3, -1, 3, 3])
            copies = 0 if length % 16 == 0 else 3 + (extra > 0)
            assert want["num_pairs"] == copies


@pytest.mark.parametrize("count", [0, 1, 2, 3])
def test_out_of_blocks_rows_keep_sharing_and_are_found_again(count):
    table = np.zeros((4, 2), np.int32)
    table[0] = [5, 6]
    c = dict(table=table, lens=np.array([20, 0, 0, 0], np.int32),
             refs=np.zeros(16, np.int32), count=count,
             stack=np.array([9, 10, 11, -1, -1, -1], np.int32))
    want = _fork(c, [0, 0, 0, 0])
    assert want["num_pairs"] == count and ("blocks" in want["flags"]) == (count < 3)
    # with blocks on the stack, the same rows are served by a call that moves nothing
    c = dict(table=want["table"], lens=want["seq_lens"], refs=want["refs"], count=3,
             stack=np.array([12, 13, 14, -1, -1, -1], np.int32))
    again = _fork(c, [0, 1, 2, 3])
    assert again["num_pairs"] == 3 - count
    assert len(set(again["table"][:, 1])) == 4 and again["refs"][5] == 3


def test_bad_sources_lengths_ids_and_counts():
    rng = np.random.default_rng(4)
    base = _tree(rng, 4, 3, 90, 6)
    assert _fork(base, [0, 12, 2, -2, 3, 3, 6, 7, 99, -1, 10, 10])["flags"] == {"metadata"}
    src = [1, 1, 1, 4, 4, -1, 6, 7, 8, 9, 9, 9]
    for bad in (-1, 16 * base["table"].shape[1] + 1, 2 ** 31 - 1, -2 ** 31):
        c = {**base, "lens": base["lens"].copy()}
        c["lens"][[0, 4]] = bad
        assert "metadata" in _fork(c, src)["flags"]
    c = {**base, "table": base["table"].copy()}
    c["lens"] = np.full(12, 37, np.int32)
    c["table"] = rng.permutation(len(base["refs"]))[:12 * 4].reshape(12, 4).astype(np.int32) \
        if len(base["refs"]) >= 48 else np.arange(48, dtype=np.int32).reshape(12, 4)
    c["refs"] = np.zeros(48, np.int32)
    c["stack"], c["count"] = np.full(80, 0, np.int32), 0
    c["table"][[0, 1, 5], [0, 2, 1]] = [-4, 48, 2 ** 31 - 1]
    assert "block id" in _fork(c, src)["flags"]
    for count in (-1, len(base["stack"]) + 1):
        assert "metadata" in _fork({**base, "count": count}, src)["flags"]


def test_counts_that_do_not_match_and_a_stack_too_small():
    """A block of two rows whose count names one holder is freed once; pushes past the
    capacity are dropped.  Both are flagged."""
    table = np.array([[3, 4], [3, 5], [6, 7]], np.int32)
    c = dict(table=table, lens=np.array([32, 32, 32], np.int32), refs=np.zeros(9, np.int32),
             stack=np.full(9, -1, np.int32), count=0)
    want = _fork(c, [-1, -1, 2])
    assert want["flags"] == {"metadata"} and want["stack"][:3].tolist() == [3, 4, 5]
    c["refs"][3] = 1
    for capacity in (0, 1, 2):
        want = _fork(c, [-1, -1, -1], capacity=capacity)
        assert want["flags"] == {"metadata"} and want["count"] == capacity


def test_no_rows_and_no_blocks():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    refs, count = torch.zeros(4, dtype=torch.int32, device="cuda"), _i32([1])
    stack = _i32([2, 3])
    mapping, pairs = pa.pa_fork_blocks(z, z.view(0, 3), z, refs, stack, count)
    assert mapping.shape == (0, 2) and int(pairs) == 0 and int(count) == 1
    lens = _i32([0, 0])
    mapping, pairs = pa.pa_fork_blocks(_i32([1, -1]), z.view(2, 0), lens, refs, stack, count)
    assert mapping.tolist() == [[-1, -1]] * 2 and int(pairs) == 0 and lens.tolist() == [0, 0]
    src, dst, moves = pa.pa_compact_blocks(z.view(0, 5), z, z.view(0, 3), z, refs, stack, count)
    assert src.shape == (0, 21) and int(count) == 1
    src, dst, moves = pa.pa_compact_blocks(z.view(2, 0), _i32([0, -1]), z.view(2, 0), lens,
                                           refs, stack, count)
    assert moves.tolist() == [0, 0] and int(count) == 1
    assert pa.pa_get_device_error() == 0


# ---- compact -----------------------------------------------------------------------
def _compact(c, keep, keep_lens, start=None, in_place=True, capacity=None):
    stack = c["stack"] if capacity is None else c["stack"][:capacity]
    table, lens, refs, st = (_i32(x) for x in (c["table"], c["lens"], c["refs"], stack))
    count = _i32([c["count"]])
    R, K = keep.shape
    src = np.full((R, K + 16), -9, np.int64)
    dst = np.full((R, K + 16), -8, np.int64)
    before = c["table"] if in_place else np.full_like(c["table"], -11)
    outs = {} if in_place else dict(
        block_tables_out=_i32(before), seq_lens_out=torch.empty_like(lens),
        extra_refs_out=torch.empty_like(refs), free_count_out=torch.empty_like(count))
    got = pa.pa_compact_blocks(
        _i32(keep), _i32(keep_lens), table, lens, refs, st, count,
        keep_start=None if start is None else _i32(start),
        src_slots=torch.from_numpy(src).cuda(), dst_slots=torch.from_numpy(dst).cuda(), **outs)
    flags = pa.pa_get_device_error()
    want = ref.compact(keep, keep_lens, start, c["table"], c["lens"], c["refs"], stack,
                       c["count"], src, dst, before)
    if not in_place:
        for t, k in ((table, "table"), (lens, "lens"), (refs, "refs")):
            np.testing.assert_array_equal(t.cpu().numpy(), c[k])
        assert int(count) == c["count"]
        table, lens, refs, count = (outs[k] for k in (
            "block_tables_out", "seq_lens_out", "extra_refs_out", "free_count_out"))
    for name, t in (("moves", got[2]), ("table", table), ("seq_lens", lens), ("refs", refs),
                    ("stack", st), ("src", got[0]), ("dst", got[1])):
        np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=name)
    assert int(count) == want["count"]
    assert flags == sum(FLAGS[f] for f in want["flags"])
    return want


def _lists(rng, c, share, tail=None):
    """Random positions to keep; tail: only among the last tokens."""
    lens = c["lens"]
    start = np.array([int(rng.integers(0, n + 1)) if tail is None else max(0, n - tail)
                      for n in lens])
    ks = [int(round(share * (n - s))) for n, s in zip(lens, start)]
    K = max(1, max(ks)) + 2
    keep = np.full((len(lens), K), 2 ** 30, np.int32)  # (past the list: never read)
    for r, (n, s, k) in enumerate(zip(lens, start, ks)):
        keep[r, :k] = s + np.sort(rng.choice(n - s, k, replace=False)) if k else []
    return keep, np.array(ks, np.int32), start.astype(np.int32)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("groups,width,hi", [(1, 1, 33), (4, 3, 60), (40, 1, 900),
                                             (9, 4, 4000), (1000, 1, 50), (1, 1, 40000)])
@pytest.mark.parametrize("share,tail", [(0.5, None), (0.05, None), (1.0, None), (0.0, None),
                                        (0.3, 40)])
def test_dropped_tokens(in_place, groups, width, hi, share, tail):
    rng = np.random.default_rng(hi + int(share * 10))
    c = _tree(rng, groups, width, hi, 4 + groups * width * hi // 16, spare=groups * hi)
    want = _compact(c, *_lists(rng, c, share, tail), in_place=in_place)
    assert not want["flags"]


def test_rows_left_as_they_are_and_truncated_ones():
    rng = np.random.default_rng(5)
    for width in (1, 3):
        c = _tree(rng, 8, width, 200, 300, spare=300)
        keep, ks, start = _lists(rng, c, 0.5)
        ks[::2] = -1
        ks[1::4] = 0                       # only the first keep_start tokens
        assert not _compact(c, keep, ks, start)["flags"]
        assert not _compact(c, keep, np.zeros_like(ks), None)["flags"]  # all dropped
        # all tokens listed: nothing changes but a shared last block
        full = np.tile(np.arange(200, dtype=np.int32), (len(ks), 1))
        assert not _compact(c, full, c["lens"])["flags"]


def test_lists_that_are_none():
    rng = np.random.default_rng(6)
    c = _tree(rng, 7, 1, 0, 60, spare=60)
    c["lens"][:] = 40
    c["table"] = np.arange(21, dtype=np.int32).reshape(7, 3)
    c["refs"] = np.zeros(60, np.int32)
    c["stack"], c["count"] = np.arange(30, 100, dtype=np.int32) % 60, 4
    keep = np.tile(np.array([3, 9, 20, 39], np.int32), (7, 1))
    keep[0, 1] = 3                         # twice the same
    keep[1, 2] = 8                         # descending
    keep[2, 3] = 40                        # past the end
    keep[3, 0] = -1
    ks = np.array([4, 4, 4, 4, 5, 4, 4], np.int32)  # 5: more than there is room for
    start = np.array([0, 0, 0, 0, 0, 4, 3], np.int32)  # 4: the list starts before it
    want = _compact(c, keep, ks, start)
    assert want["flags"] == {"metadata"}
    assert want["seq_lens"].tolist() == [40] * 6 + [7]
    for bad in (-1, 41, 2 ** 31 - 1):
        start[6] = bad
        assert _compact(c, keep, np.maximum(ks, 0) * 0 + 1, start)["flags"] == {"metadata"}
    c["lens"][[2, 5]] = [-1, 49]
    assert "metadata" in _compact(c, keep, np.full(7, 2, np.int32))["flags"]


@pytest.mark.parametrize("free", [0, 1, 2, 3, 6])
def test_blocks_held_by_others_are_replaced_while_the_stack_lasts(free):
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    refs = np.zeros(32, np.int32)
    refs[[0, 1, 2, 5, 9, 11]] = [1, 2, 1, 1, 1, 3]
    c = dict(table=table, lens=np.array([64, 50, 49], np.int32), refs=refs,
             stack=np.arange(20, 32, dtype=np.int32), count=free)
    keep = np.array([[1] + list(range(17, 50)), list(range(16, 50)), list(range(2, 36))],
                    np.int32)
    want = _compact(c, keep, np.array([34, 34, 34], np.int32))
    assert ("blocks" in want["flags"]) == (free < 5)
    # ids on the stack that are none
    c["stack"] = np.full(12, 32, np.int32)
    _compact(c, keep, np.array([34, 34, 34], np.int32))


def test_a_block_of_two_rows_that_both_drop_tokens():
    """Both rows get a block of their own; the old one goes back once."""
    c = dict(table=np.array([[1, 2, 3], [1, 2, 4]], np.int32),
             lens=np.array([40, 41], np.int32), refs=np.zeros(16, np.int32),
             stack=np.array([10, 11, 12, 13, 14, 15, 0, 0, 0], np.int32), count=6)
    c["refs"][[1, 2]] = 1
    keep = np.array([list(range(1, 38)), list(range(3, 40))], np.int32)
    want = _compact(c, keep, np.array([37, 37], np.int32))
    assert not want["flags"] and want["count"] == 4
    assert want["stack"][2:4].tolist() == [1, 2]
