"""pa_fork_blocks with ids on the stack that are no blocks: the row that pops one holds it
and no longer the shared block, exactly as the plain loop has it."""
import numpy as np
import pytest

from tests import test_gpu_fork as fork

pytestmark = fork.pytestmark


def _shared(rng, groups, width):
    """Rows that share all but a partly filled last block."""
    c = fork._tree(rng, groups, width, 0, 0)
    R, full = groups * width, 3
    lens = np.full(R, 16 * full + 5)
    table = np.full((R, full + 2), -7)
    NB = groups * full + R + 2 * R
    for r in range(R):
        table[r, :full] = r // width * full + np.arange(full)
        table[r, full] = groups * full + r
    extra = np.zeros(NB, np.int64)
    extra[:groups * full] = width - 1
    stack = np.full(4 * R, -1)
    stack[:2 * R] = groups * full + R + np.arange(2 * R)
    c.update(table=table.astype(np.int32), lens=lens.astype(np.int32),
             refs=extra.astype(np.int32), stack=stack.astype(np.int32), count=2 * R)
    return c, NB


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("groups,width", [(1, 4), (16, 4), (200, 8)])
def test_popped_ids_that_are_no_blocks(in_place, groups, width):
    """All rows of a group on the first one's last block, no row released (s = r): each but
    the first pops an id, every third of them no block.  Then rows released in the same
    call, whose blocks lie above such ids and are popped; and a stack of only such ids that
    runs out."""
    rng = np.random.default_rng(groups)
    c, NB = _shared(rng, groups, width)
    R = groups * width
    # all rows take the first one's block: a state in which the copies are still to come
    first = np.repeat(np.arange(groups) * width, width)
    last = c["table"][:, 3].copy()
    c["table"][:, 3] = last[first]
    c["refs"][last[first[::width]]] = width - 1
    top = c["count"]
    for bad in (-1, NB, 2 ** 31 - 1, -2 ** 31, -5):
        d = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
        d["stack"][top - 1:top - R:-3] = bad
        want = fork._fork(d, np.arange(R), in_place)
        assert want["flags"] == {"block id"} and want["num_pairs"] == R - groups
    # and with rows released in the same call: their blocks are popped first
    d = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
    d["table"][:, 3] = last
    d["refs"][last] = 0
    d["stack"][:top] = -1
    sources = first.copy()
    sources[width // 2::width] = -1
    want = fork._fork(d, sources, in_place)
    assert not want["flags"]
    d["count"] = 3
    sources = np.arange(R)
    d["table"][1::width, 3] = d["table"][0::width, 3]
    d["refs"][last[0::width]] = 1
    want = fork._fork(d, sources, in_place)
    assert "block id" in want["flags"]
