"""The calls of several hypotheses as the first ones that a process makes of the library,
inside a capture: what they look up of the device must be allowed there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

START = """
import torch
import paged_kv_cache_82_gb300 as pa
def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
state = dict(block_tables=i32([0, 1], [2, 3]), seq_lens=i32(20, 20), extra_refs=i32(*[0] * 8),
             free_blocks=i32(4, 5, 6, 7, 0, 0, 0, 0), free_count=i32(4))
work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
pool = torch.arange(2 * 8 * 2 * 16 * 64, device="cuda").bfloat16().view(2, 8, 2, 16, 64)
k, v = pool.clone(), pool.clone() + 1
i64 = lambda *x: torch.tensor(x, dtype=torch.int64, device="cuda")
x = (torch.arange(1000, device="cuda").float() / 500).repeat(4, 1)
cum, sources, one, kept = torch.zeros(1, 4, device="cuda"), i32(0, 0), i32(1), i32([2], [3])
pairs, src, dst = i64([1, 5]), i64([17], [40]), i64([2], [33])
ones, starts = i32(1, 1), i32(1, 1)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = CALL
graph.replay()
torch.cuda.synchronize()
assert pa.pa_get_device_error() == 0
"""
CALLS = {
    "beam": ("pa.pa_beam_select(x, cum, 2, workspace=work)",
             "assert out[2].tolist() == [[999, 999]] and out[1].tolist() == [[0, 1]], out"),
    "fork": ("pa.pa_fork_blocks(sources, workspace=work, **state)",
             "assert state['block_tables'].tolist() == [[0, 1], [0, 3]], state"),
    "copy": ("pa.pa_copy_blocks_layers(k, v, pairs, one)",
             "assert torch.equal(k[:, 5], pool[:, 1]) and torch.equal(v[:, 5], pool[:, 1] + 1)"),
    "compact": ("pa.pa_compact_blocks(kept, ones, keep_start=starts, workspace=work, **state)",
                "assert state['seq_lens'].tolist() == [2, 2], state"),
    "move": ("pa.pa_move_tokens(k, v, src, dst, ones)",
             "assert torch.equal(k[:, 0, :, 2], pool[:, 1, :, 1]) and "
             "torch.equal(v[:, 2, :, 1], pool[:, 2, :, 8] + 1)"),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_first_call_of_a_process_captured(name):
    call, check = CALLS[name]
    program = START.replace("CALL", call) + check + "\n"
    done = subprocess.run([sys.executable, "-c", program], cwd=ROOT, timeout=240,
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-3000:]
