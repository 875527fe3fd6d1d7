"""The sparse decode step's operators together, as a serving loop runs them:
metadata, norm + rotation + cache write, bounds, selection, attention -- eager
and as one captured graph replayed step by step, on two streams at once, and
with a workspace that two graphs share."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, K = 8, 2, 128, 5
SPAN = 600


class Loop:
    """A paged cache and the state of a few requests, all on the GPU."""

    def __init__(self, seed, prompts, cache="bf16", pad=2, workspaces=None):
        self.rng = np.random.default_rng(seed)
        B = len(prompts)
        self.cache, self.B, self.prompts = cache, B, prompts
        NB, M = 120, 40
        i32 = dict(dtype=torch.int32, device="cuda")
        self.NB = NB
        ids = self.rng.permutation(NB).astype(np.int32)
        self.free = torch.from_numpy(ids).cuda()
        self.count = torch.tensor([NB], **i32)
        self.table = torch.full((B, M), -1, **i32)
        self.lens = torch.zeros(B, **i32)
        dt = torch.uint8 if cache == "e4m3" else torch.bfloat16
        nan = 0x7F if cache == "e4m3" else float("nan")
        self.kc = torch.full((NB, HKV, 16, D), nan, dtype=dt, device="cuda")
        self.vc = self.kc.clone()
        self.sc = (0.02, 0.01) if cache == "e4m3" else (1.0, 1.0)
        self.bounds = torch.zeros(NB, HKV, pa.bounds_bytes(D), dtype=torch.uint8, device="cuda")
        freq = 10000.0 ** (-np.arange(0, D, 2) / D)
        ang = np.arange(SPAN)[:, None] * freq
        self.cs = torch.from_numpy(
            np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
        self.w = [torch.from_numpy(self.rng.uniform(0.5, 1.5, D).astype(np.float32)
                                   ).bfloat16().cuda() for _ in range(2)]
        self.ws = workspaces or [torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
                                 for _ in range(2)]
        self.pad = pad

    def buffers(self, T):
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(T=T, qkv=torch.zeros(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16,
                                         device="cuda"),
                    new=torch.zeros(self.B, **i32), qsl=torch.zeros(self.B + 1, **i32),
                    pos=torch.zeros(T, **i32),
                    slots=torch.zeros(T, dtype=torch.int64, device="cuda"),
                    q=torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda"),
                    sel=torch.full((T, HKV, K), -7, **i32), cnt=torch.full((T, HKV), -7, **i32),
                    out=torch.full((T, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda"))

    def step(self, b, max_q, stream=None):
        """One step on the current stream: state updated in place."""
        T, qkv = b["T"], b["qkv"]
        pa.pa_build_step(b["new"], self.lens, self.table, self.free, self.count, self.NB, T,
                         seq_lens=self.lens, query_start_loc=b["qsl"], positions=b["pos"],
                         slot_mapping=b["slots"], free_count_out=self.count, stream=stream)
        pa.pa_norm_rope_and_cache(
            qkv[:, :HQ * D].unflatten(1, (HQ, D)),
            qkv[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)),
            qkv[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)), self.kc, self.vc, b["slots"],
            b["pos"], self.cs, *self.w, k_scale=self.sc[0], v_scale=self.sc[1], q_out=b["q"],
            stream=stream)
        m = (self.table, self.lens, b["qsl"])
        pa.pa_summarise_blocks(self.kc, self.bounds, *m, T, max_q, SPAN, stream=stream)
        pa.pa_select_blocks(b["q"], self.bounds, *m, max_q, SPAN, K, 1, 1, selected=b["sel"],
                            num_selected=b["cnt"], workspace=self.ws[0], stream=stream)
        pa.pa_attention_selected(b["q"], self.kc, self.vc, *m, max_q, SPAN, D ** -0.5, b["sel"],
                                 b["cnt"], *self.sc, out=b["out"], workspace=self.ws[1],
                                 stream=stream)

    def fill(self, b, new):
        x = self.rng.standard_normal((b["T"], (HQ + 2 * HKV) * D)) * 2
        b["qkv"].copy_(torch.from_numpy(x.astype(np.float32)))
        b["new"].copy_(torch.tensor(new, dtype=torch.int32))
        b["out"].fill_(7)  # rows of an earlier, longer step

    def check(self, b):
        """The step's results from the cache, queries and tables it left."""
        md = dict(query_start_loc=b["qsl"].cpu().numpy(), seq_lens=self.lens.cpu().numpy(),
                  block_tables=self.table.cpu().numpy())
        T = int(md["query_start_loc"][-1])
        k = ref.decode_pages(self.kc, self.cache, D)
        v = ref.decode_pages(self.vc, self.cache, D)
        hi, lo, sc = ref.records(self.bounds, D)
        for r in range(self.B):
            L = int(md["seq_lens"][r])
            for blk in range(-(-L // 16)):
                p = md["block_tables"][r, blk]
                for h in range(HKV):
                    w = ref.bounds_of(k[p, h, :min(16, L - 16 * blk)])
                    np.testing.assert_array_equal(hi[p, h], w[0])
                    np.testing.assert_array_equal(lo[p, h], w[1])
                    assert sc[p, h] == w[2]
        # keys and values of this step are where the metadata says
        qn, _ = ref.norm_rope(
            b["qkv"][:T, :HQ * D].float().cpu().numpy().reshape(T, HQ, D),
            self.w[0].float().cpu().numpy(), 1e-6, self.cs.cpu().numpy(),
            b["pos"].cpu().numpy()[:T], False)
        q = b["q"].double().cpu().numpy()
        assert np.abs(q[:T] - qn).max() <= 2 ** -7 * np.abs(qn).max()
        for t, r, p in ref.tokens_of(md):
            assert int(b["pos"][t]) == p
            slot = int(md["block_tables"][r, p // 16]) * 16 + p % 16
            assert int(b["slots"][t]) == slot
        want = ref.select(q.astype(np.float32), hi, lo, sc, md, HQ // HKV, K, 1, 1)
        for (t, h), blocks in want.items():
            assert b["sel"][t, h].tolist() == blocks + [-1] * (K - len(blocks))
            assert int(b["cnt"][t, h]) == len(blocks)
        ref_out, mag, qk = ref.attend(q, k, v, md, want, HQ // HKV, D ** -0.5, *self.sc)
        tol = ref.attend_tolerance(ref_out, mag, qk, "bf16",
                                   "f16" if self.cache == "e4m3" else "bf16")
        got = b["out"].float().cpu().double().numpy()
        assert (np.abs(got[:T] - ref_out[:T]) <= tol[:T]).all()
        assert (got[T:] == 7).all()  # rows behind the last request

    def prefill(self):
        b = self.buffers(sum(self.prompts) + self.pad)
        self.fill(b, self.prompts)
        self.step(b, max(self.prompts))
        return b


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prompt_then_captured_decode_steps(cache):
    loop = Loop(1, [70, 1, 33, 200], cache)
    loop.check(loop.prefill())
    b = loop.buffers(loop.B + loop.pad)
    eager = 3
    for _ in range(eager):
        loop.fill(b, [1] * loop.B)
        loop.step(b, 1)
        loop.check(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        loop.step(b, 1)
    for i in range(40):
        # now and then a request that has nothing to do in the step
        loop.fill(b, [1, 1, int(i % 5 != 2), 1])
        g.replay()
        if i % 8 == 7 or i == 2:
            loop.check(b)
    assert pa.pa_get_device_error() == 0
    assert loop.lens.tolist() == [70 + 43, 1 + 43, 33 + 43 - 8, 200 + 43]


def test_chunks_and_drafted_tokens_in_one_step():
    loop = Loop(2, [90, 20, 5])
    loop.check(loop.prefill())
    b = loop.buffers(64)
    for new in ([1, 40, 3], [0, 1, 50], [4, 4, 4]):
        loop.fill(b, new)
        loop.step(b, 50)
        loop.check(b)
    assert pa.pa_get_device_error() == 0


def test_two_loops_on_two_streams_at_once():
    loops = [Loop(3, [60, 120]), Loop(4, [150, 10])]
    streams = [torch.cuda.Stream() for _ in loops]
    bufs = []
    for lp in loops:
        lp.prefill()
        bufs.append(lp.buffers(2))
    torch.cuda.synchronize()
    for _ in range(12):
        for lp, b in zip(loops, bufs):
            lp.fill(b, [1, 1])
        torch.cuda.synchronize()
        for lp, b, s in zip(loops, bufs, streams):
            lp.step(b, 1, stream=s)
        torch.cuda.synchronize()
    for lp, b in zip(loops, bufs):
        lp.check(b)
    assert pa.pa_get_device_error() == 0


def test_two_graphs_that_share_a_workspace():
    """Replayed one after the other on one stream, with the previous graph's
    leavings in it."""
    ws = [torch.full((1 << 23,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    loops = [Loop(5, [180, 30], workspaces=ws), Loop(6, [20, 250], "e4m3", workspaces=ws)]
    bufs, graphs = [], []
    for lp in loops:
        lp.prefill()
        b = lp.buffers(2)
        lp.fill(b, [1, 1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lp.step(b, 1)
        bufs.append(b)
        graphs.append(g)
    for _ in range(5):
        for lp, b, g in zip(loops, bufs, graphs):
            lp.fill(b, [1, 1])
            g.replay()
    for lp, b in zip(loops, bufs):
        lp.check(b)
    assert pa.pa_get_device_error() == 0


def test_running_out_of_blocks_ends_the_loop_cleanly():
    """The request that finds no block gets no token; the others go on, and a
    released block lets it continue."""
    loop = Loop(7, [16, 40])
    loop.prefill()
    loop.count.fill_(0)
    b = loop.buffers(2)
    loop.fill(b, [1, 1])
    loop.step(b, 1)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_NO_BLOCKS
    # the first request needed a block: neither it nor the one after it runs
    assert loop.lens.tolist() == [16, 40] and b["slots"].tolist() == [-1, -1]
    assert (b["out"] == 7).all()
    loop.count.fill_(1)
    loop.fill(b, [1, 1])
    loop.step(b, 1)
    loop.check(b)
    assert pa.pa_get_device_error() == 0 and int(loop.count) == 0
