"""pa_build_step on the GPU against a plain loop, exactly."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref

pytestmark = pytest.mark.gpu

FLAGS = {"metadata": pa.PA_DEV_ERR_METADATA, "blocks": pa.PA_DEV_ERR_NO_BLOCKS,
         "block id": pa.PA_DEV_ERR_BLOCK_ID}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda").reshape(-1)


def _case(rng, lens, width=None, free=None, pad=0, num_blocks=None):
    """lens: (computed, new) per request."""
    have = [-(-max(c, 0) // 16) for c, _ in lens]
    want = sum(max(0, -(-(c + n) // 16) - -(-c // 16)) for c, n in lens if c >= 0 and n >= 0)
    free = want + 3 if free is None else free
    width = width or max([1] + [-(-(c + max(n, 0)) // 16) for c, n in lens]) + 2
    nb = num_blocks or sum(have) + free + 5
    ids = rng.permutation(max(nb, sum(have) + free)).astype(np.int32)
    table = rng.integers(-9, -1, size=(len(lens), width)).astype(np.int32)  # never read
    k = 0
    for r, h in enumerate(have):
        h = min(h, width)
        table[r, :h] = ids[k:k + h]
        k += h
    stack = ids[k:k + free]
    T = sum(max(n, 0) for _, n in lens) + pad
    return dict(query_lens=[n for _, n in lens], computed_lens=[c for c, _ in lens],
                table=table, stack=stack, T=T, nb=nb)


def _run(c, in_place=False, T=None, count=None):
    T = c["T"] if T is None else T
    count = len(c["stack"]) if count is None else count
    table = torch.from_numpy(c["table"].copy()).cuda()
    done, cnt = _i32(c["computed_lens"]), _i32([count])
    stack = _i32(c["stack"]) if len(c["stack"]) else torch.zeros(0, dtype=torch.int32,
                                                                 device="cuda")
    got = pa.pa_build_step(_i32(c["query_lens"]), done, table, stack, cnt, c["nb"], T,
                           seq_lens=done if in_place else None,
                           free_count_out=cnt if in_place else None)
    flags = pa.pa_get_device_error()
    want = ref.build_step(c["query_lens"], c["computed_lens"], c["table"], c["stack"],
                          count, T, c["nb"])
    for name, t in zip(("seq_lens", "query_start_loc", "positions", "slot_mapping"), got):
        assert t.cpu().numpy().dtype == want[name].dtype, name
        np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=name)
    np.testing.assert_array_equal(table.cpu().numpy(), want["table"])
    assert int(got[4]) == want["free_count"]
    assert flags == sum(FLAGS[f] for f in want["flags"])
    return want


CASES = {
    "first_token": [(0, 1)],
    "prompts": [(0, 5), (0, 16), (0, 17), (0, 1)],
    "block_edges": [(15, 1), (16, 1), (17, 1), (31, 2), (32, 0), (0, 0), (1, 0)],
    "chunk_mid_block": [(7, 100), (16, 48), (33, 15), (1, 1)],
    "empty_rows_between": [(3, 0), (0, 0), (5, 2), (9, 0), (0, 3), (4, 0)],
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_small_steps(name, in_place):
    rng = np.random.default_rng(len(name))
    want = _run(_case(rng, CASES[name], pad=5), in_place)
    assert not want["flags"]


@pytest.mark.parametrize("B,hi,chunks", [(64, 4096, 0), (1023, 3000, 2), (1024, 100, 0),
                                         (1025, 700, 5), (5000, 40, 1), (16384, 9, 0)])
def test_large_steps(B, hi, chunks):
    """One and several scan rounds, one to eight CTAs, shared memory past 48 KB."""
    rng = np.random.default_rng(B)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, hi, B), rng.integers(0, 3, B))]
    for i in range(chunks):
        lens[int(rng.integers(0, B))] = (int(rng.integers(0, hi)), 1777)
    _run(_case(rng, lens, pad=int(rng.integers(0, 90))))


def test_matches_the_host_builder():
    """The same arrays as the host builder's from the same requests."""
    from workloads import Request
    rng = np.random.default_rng(3)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, 300, 40), rng.integers(1, 60, 40))]
    c = _case(rng, lens)
    want = _run(c)
    reqs = [Request([int(b) for b in want["table"][r, :-(-(a + n) // 16)]], a, n)
            for r, (a, n) in enumerate(lens)]
    md = oracle.step_metadata(reqs)
    for k in ("seq_lens", "query_start_loc", "slot_mapping"):
        np.testing.assert_array_equal(want[k], md[k])


@pytest.mark.parametrize("free", [0, 1, 2, 5, 6])
def test_out_of_blocks_stops_the_step_there(free):
    rng = np.random.default_rng(free)
    lens = [(16, 1), (10, 2), (32, 33), (5, 1), (16, 1)]  # needs 1, 0, 3, 0, 1
    want = _run(_case(rng, lens, free=free), in_place=True)
    assert ("blocks" in want["flags"]) == (free < 5)


@pytest.mark.parametrize("T", [0, 1, 3, 36, 37])
def test_tokens_beyond_the_arrays_stop_the_step(T):
    rng = np.random.default_rng(T)
    want = _run(_case(rng, [(16, 1), (10, 2), (32, 33), (5, 1)]), T=T)
    assert ("metadata" in want["flags"]) == (T < 37)


def test_bad_lengths_ids_and_counts():
    rng = np.random.default_rng(8)
    # a request past its table, a negative length, a negative count of tokens
    c = _case(rng, [(3, 2), (16 * 6, 1), (-1, 4), (20, -2), (7, 4)], width=6, free=9)
    assert _run(c)["flags"] == {"metadata"}
    # a stack height outside the stack: nothing is popped
    for count in (-1, 10):
        c = _case(rng, [(3, 2), (16, 1)], free=9)
        assert _run(c, count=count)["flags"] == {"metadata", "blocks"}
    # ids outside the pool, in the table and on the stack
    c = _case(rng, [(3, 2), (16, 1), (40, 20)], free=9)
    c["stack"][-1] = c["nb"]
    c["table"][2, 2] = -3
    assert _run(c)["flags"] == {"block id"}


def test_no_requests_and_no_tokens():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = pa.pa_build_step(z, z, z.view(0, 4), _i32([7]), _i32([1]), 8, 3)
    assert got[1].tolist() == [0] and got[2].tolist() == [0, 0, 0]
    assert got[3].tolist() == [-1, -1, -1] and int(got[4]) == 1
    got = pa.pa_build_step(_i32([0]), _i32([0]), torch.zeros(1, 0, dtype=torch.int32,
                                                             device="cuda"),
                           z, _i32([0]), 8, 0)
    assert got[0].tolist() == [0] and got[1].tolist() == [0, 0]
    assert pa.pa_get_device_error() == 0


def test_captured_loop_updates_its_state_in_place():
    """200 replays of one captured step: 200 tokens per request, each block
    popped once, the same as the plain loop's."""
    rng = np.random.default_rng(5)
    lens = [(int(c), 1) for c in rng.integers(0, 100, 33)]
    c = _case(rng, lens, width=24, free=33 * 13 + 7)
    table, done = torch.from_numpy(c["table"].copy()).cuda(), _i32(c["computed_lens"])
    cnt, stack, one = _i32([len(c["stack"])]), _i32(c["stack"]), _i32(c["query_lens"])
    bufs = dict(query_start_loc=torch.empty(34, dtype=torch.int32, device="cuda"),
                positions=torch.empty(40, dtype=torch.int32, device="cuda"),
                slot_mapping=torch.empty(40, dtype=torch.int64, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pa.pa_build_step(one, done, table, stack, cnt, c["nb"], 40, seq_lens=done,
                         free_count_out=cnt, **bufs)
    state = dict(computed=np.array(c["computed_lens"]), table=c["table"].copy(),
                 count=len(c["stack"]))
    for _ in range(200):
        g.replay()
        w = ref.build_step(c["query_lens"], state["computed"], state["table"], c["stack"],
                           state["count"], 40, c["nb"])
        state = dict(computed=w["seq_lens"], table=w["table"], count=w["free_count"])
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    np.testing.assert_array_equal(table.cpu().numpy(), state["table"])
    np.testing.assert_array_equal(done.cpu().numpy(), state["computed"])
    np.testing.assert_array_equal(bufs["slot_mapping"].cpu().numpy(), w["slot_mapping"])
    assert int(cnt) == state["count"]
