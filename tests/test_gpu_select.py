"""pa_summarise_blocks and pa_select_blocks on the GPU against plain loops,
exactly: their results are whole numbers by definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
import workloads
from paged_kv_cache_82_gb300.metadata import build_step_metadata
from tests import _sparse_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def step(lens, Hq, Hkv, D, dtype="bf16", cache=None, seed=1):
    """lens: (L, n) per request; the cache holds all keys, other slots NaN."""
    need = sum(-(-L // 16) for L, _ in lens)
    wl = workloads.decode_step(
        "sel", seed, seq_lens=[L for L, _ in lens], q_lens=[n for _, n in lens],
        num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, num_blocks=need + 5, dtype=dtype,
        cache_dtype=cache or dtype, write_new=False,
        k_scale=0.5 if cache in ("e4m3", "nvfp4") else 1.0,
        v_scale=0.25 if cache in ("e4m3", "nvfp4") else 1.0)
    md = build_step_metadata(wl.requests)
    dev = {k: torch.from_numpy(md[k]).cuda()
           for k in ("block_tables", "seq_lens", "query_start_loc")}
    return wl, md, dev


def meta(dev):
    return dev["block_tables"], dev["seq_lens"], dev["query_start_loc"]


LENS = [(1, 1), (15, 1), (16, 1), (17, 1), (40, 9), (33, 33), (300, 270), (64, 0), (128, 16)]


@pytest.mark.parametrize("cache,D", [("bf16", 128), ("f16", 64), ("f32", 128), ("f32", 64),
                                     ("e4m3", 128), ("e4m3", 64), ("int4", 128),
                                     ("nvfp4", 64), ("int4", 64), ("nvfp4", 128)])
def test_summaries(cache, D):
    dtype = cache if cache in DT else "bf16"
    wl, md, dev = step(LENS, 6, 3, D, dtype, cache)
    NB = wl.k_cache.shape[0]
    rng = np.random.default_rng(1)
    init = torch.from_numpy(rng.integers(0, 256, (NB, 3, pa.bounds_bytes(D)), dtype=np.uint8))
    got = init.clone().cuda()
    pa.pa_summarise_blocks(wl.k_cache.cuda(), got, *meta(dev), wl.num_tokens,
                           md["max_query_len"], md["max_seq_len"], cache_dtype=cache)
    assert pa.pa_get_device_error() == 0
    k = ref.decode_pages(wl.k_cache, cache, D)
    want = init.numpy().copy()
    for r, (L, n) in enumerate(LENS):
        for b in range((L - n) // 16, -(-L // 16)) if n else []:
            blk = md["block_tables"][r, b]
            for h in range(3):
                hi, lo, s = ref.bounds_of(k[blk, h, :min(16, L - 16 * b)])
                want[blk, h, :D] = hi.view(np.uint8)
                want[blk, h, D:2 * D] = lo.view(np.uint8)
                want[blk, h, 2 * D:] = 0
                want[blk, h, 2 * D:2 * D + 4] = np.frombuffer(s.tobytes(), np.uint8)
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_summaries_of_odd_values():
    """Zeros, NaN, infinities, values near fp32's ends, one sign only."""
    D, f = 64, np.float32
    keys = np.random.default_rng(2).standard_normal((8, 16, D)).astype(f)
    keys[0] = 0
    keys[1, 3, :] = np.nan
    keys[2, :, 5] = np.nan
    keys[3, 0, 7], keys[3, 1, 8] = np.inf, -np.inf
    keys[4] = np.abs(keys[4]) + 1
    keys[5] *= f(1e-38)
    keys[6] *= f(3e37)
    keys[7, :, :] = -2.5
    kc = torch.from_numpy(keys).view(8, 1, 16, D).cuda()
    got = torch.zeros(8, 1, pa.bounds_bytes(D), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    pa.pa_summarise_blocks(kc, got, torch.arange(8, **i32)[None].contiguous(),
                           torch.tensor([128], **i32), torch.tensor([0, 128], **i32), 128,
                           128, 128)
    assert pa.pa_get_device_error() == 0
    hi, lo, s = ref.records(got, D)
    for b in range(8):
        w = ref.bounds_of(keys[b].astype(np.float64))
        np.testing.assert_array_equal(hi[b, 0], w[0])
        np.testing.assert_array_equal(lo[b, 0], w[1])
        assert s[b, 0] == w[2]
        # The codes bound the keys up to the roundings.  s is off big / 127 by
        # at most 2^-24 of it and 2^-150 (subnormal s), so the cut at 127 takes
        # at most 2^-24 big + 127 x 2^-150; the quotient under the ceiling is
        # off by 2^-24 of itself, |x| <= big: together 2^-23 big + 2^-143.
        # (Signs differ, so the slack is added, not multiplied.)
        x = np.where(np.isfinite(keys[b]), keys[b], 0).astype(np.float64)
        sd = float(s[b, 0])
        slack = 2.0 ** -23 * 127 * sd * (1 + 1e-6) + 2.0 ** -142
        top, low = hi[b, 0] * sd + slack, lo[b, 0] * sd - slack
        ok = np.isfinite(keys[b])
        assert (np.where(ok, x, low) <= top).all() and (np.where(ok, x, top) >= low).all()


def _select(wl, dev, md, bounds, K, first, last, q=None, T=None, **kw):
    q = wl.q.cuda() if q is None else q
    return pa.pa_select_blocks(q, bounds, *meta(dev), md["max_query_len"],
                               md["max_seq_len"], K, keep_first=first, keep_last=last, **kw)


def _random_bounds(NB, Hkv, D, seed, ties=False):
    rng = np.random.default_rng(seed)
    b = np.zeros((NB, Hkv, 2 * D + 16), dtype=np.uint8)
    hi = rng.integers(0, 3, (NB, Hkv, D)) if ties else rng.integers(-90, 128, (NB, Hkv, D))
    lo = -hi if ties else np.minimum(hi, rng.integers(-127, 90, (NB, Hkv, D)))
    if ties:  # few different blocks: many equal scores
        pick = rng.integers(0, 3, (NB, 1))
        hi, lo = hi[pick, np.arange(Hkv)], lo[pick, np.arange(Hkv)]
    b[..., :D] = hi.astype(np.int8).view(np.uint8)
    b[..., D:2 * D] = lo.astype(np.int8).view(np.uint8)
    sc = np.full((NB, Hkv), 0.01, np.float32) if ties else rng.uniform(
        0.0, 0.05, (NB, Hkv)).astype(np.float32)
    sc[::7] = sc[::7] if ties else 0  # blocks of zero keys
    b[..., 2 * D:2 * D + 4] = sc[..., None].view(np.uint8)
    return torch.from_numpy(b).cuda()


CASES = {
    # lens, Hq, Hkv, D, dtype, K, first, last
    "decode": ([(L, 1) for L in (1, 16, 17, 48, 49, 333, 1000, 5003)], 32, 8, 128, "bf16",
               7, 1, 2),
    "one_kept": ([(700, 1), (31, 1), (16, 1)], 8, 8, 128, "f16", 1, 0, 1),
    "all_kept": ([(700, 1), (65, 1)], 8, 2, 64, "f32", 6, 2, 4),
    "chunk": ([(900, 130), (40, 40), (77, 1), (64, 0), (300, 5)], 12, 3, 128, "bf16", 9, 1, 1),
    "group8": ([(3000, 2), (4096, 1)], 64, 8, 128, "bf16", 33, 0, 3),
    "group16_d64": ([(2500, 1), (640, 3)], 32, 2, 64, "f16", 20, 3, 1),
    "group20": ([(2500, 1)], 20, 1, 64, "bf16", 21, 1, 1),
    "mha": ([(1200, 1), (2222, 1)], 9, 9, 128, "bf16", 30, 1, 1),
    "wide_k": ([(40000, 1), (9000, 1)], 4, 1, 128, "bf16", 700, 1, 2),
}


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_selection(name, ties):
    lens, Hq, Hkv, D, dtype, K, first, last = CASES[name]
    wl, md, dev = step(lens, Hq, Hkv, D, dtype)
    bounds = _random_bounds(wl.k_cache.shape[0], Hkv, D, len(name), ties)
    sel, cnt = _select(wl, dev, md, bounds, K, first, last)
    assert pa.pa_get_device_error() == 0
    hi, lo, sc = ref.records(bounds, D)
    want = ref.select(wl.q.float().numpy(), hi, lo, sc, md, Hq // Hkv, K, first, last)
    sel, cnt = sel.cpu().numpy(), cnt.cpu().numpy()
    assert len(want) == wl.num_tokens * Hkv
    for (t, h), blocks in want.items():
        assert cnt[t, h] == len(blocks)
        np.testing.assert_array_equal(sel[t, h], blocks + [-1] * (K - len(blocks)))


def test_a_score_bounds_the_blocks_keys():
    """With q = sq qc + d, |d| <= sq / 2 per channel (rounding to codes), and
    keys between the codes times s (up to 2^-23 of the largest, above):
    max_j <q, k_j> <= sq (score + 2^-23 s 127 sum |qc|) + (sq / 2) sum_d
    max_j |k_jd|.  So a selection by score leaves out no block by more than
    the query's own rounding.  The blocks selected are those of the scores."""
    lens = [(4000, 1), (1500, 1)]
    wl, md, dev = step(lens, 8, 8, 128)
    NB = wl.k_cache.shape[0]
    bounds = torch.zeros(NB, 8, pa.bounds_bytes(128), dtype=torch.uint8, device="cuda")
    whole = torch.tensor([0, 4000, 5500], dtype=torch.int32, device="cuda")
    pa.pa_summarise_blocks(wl.k_cache.cuda(), bounds, dev["block_tables"], dev["seq_lens"],
                           whole, 5500, 4000, 4000)
    k = ref.decode_pages(wl.k_cache, "bf16", 128)
    q = wl.q.clone()
    for r, (L, _) in enumerate(lens):  # a query close to one far key
        at = L // 3
        q[r] = wl.k_cache[md["block_tables"][r, at // 16], :, at % 16] * 3
    sel, _ = _select(wl, dev, md, bounds, 4, 0, 1, q=q.cuda())
    assert pa.pa_get_device_error() == 0
    hi, lo, sc = ref.records(bounds, 128)
    want = ref.select(q.float().numpy(), hi, lo, sc, md, 1, 4, 0, 1)
    for r, (L, _) in enumerate(lens):
        blk = md["block_tables"][r, :L // 16]
        for h in range(8):
            assert sel[r, h].tolist() == want[r, h]
            x = q[r, h].double().numpy()
            sq = float(np.float32(np.abs(x).max()) / np.float32(127))
            qc = np.rint(x / sq)
            kb = k[blk, h]
            s = sc[blk, h].astype(np.float64)
            score = s * (np.maximum(qc, 0) @ hi[blk, h].T + np.minimum(qc, 0) @ lo[blk, h].T)
            best = (kb @ x).max(-1)
            slack = 2.0 ** -22 * s * 127 * np.abs(qc).sum()
            reach = np.abs(kb).max(1).sum(-1) * (sq / 2) * (1 + 1e-5)
            assert (best <= sq * (score + slack) + reach).all()


def test_odd_queries():
    """Zero, infinite and NaN queries: defined selections, no flag."""
    wl, md, dev = step([(900, 1)] * 4, 8, 2, 64, "f32")
    bounds = _random_bounds(wl.k_cache.shape[0], 2, 64, 4)
    q = wl.q.clone()
    q[0] = 0
    q[1, 0, 3] = float("inf")
    q[2, 1, :] = 3e38
    q[3, 2, 5] = float("nan")
    sel, cnt = _select(wl, dev, md, bounds, 5, 1, 1, q=q.cuda())
    assert pa.pa_get_device_error() == 0
    # no order among equal zero scores: the lowest blocks
    for t in (0, 1):
        want = [0, 1, 2, 3, 56]
        assert sel[t, 0].tolist() == want
    assert sel[0, 1].tolist() == [0, 1, 2, 3, 56]
    s = sel.cpu()
    assert (s.diff(dim=-1) > 0).all() and int(cnt.min()) == 5


def _order(x):
    """fp32 scores as whole numbers of their order, a NaN above all."""
    u = (x + np.float32(0)).view(np.uint32).astype(np.int64)
    key = np.where(u >> 31, 0xFFFFFFFF - u, u | 0x80000000)
    return np.where(np.isnan(x), 0xFFFFFFFE, key)


@pytest.mark.parametrize("L", [4800, 40 * 1024, 160 * 1024])
def test_records_of_any_bytes(L):
    """Records that were never written: any codes and scales, NaN and infinities
    among them.  A list is that of the scores all the same, a NaN's above all,
    and nothing is written past a list's K entries."""
    n = L // 16
    rng = np.random.default_rng(n)
    raw = rng.integers(0, 256, (n, 2, 2 * 64 + 16), dtype=np.uint8)
    raw[rng.integers(0, n, 3), :, 128:132] = (0, 0, 0xC0, 0x7F)  # NaN
    raw[rng.integers(0, n, 3), :, 128:132] = (0, 0, 0x80, 0x7F)  # infinite
    bounds = torch.from_numpy(raw).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = rng.permutation(n).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((1, 4, 64)).astype(np.float32))
    hi, lo, sc = ref.records(bounds, 64)
    x = q.numpy()[0].reshape(2, 2, 64)
    for K in (2, 3, 5, 9, 60, 290):
        out = torch.full((2 * K + 4096,), -77, **i32)
        sel, _ = pa.pa_select_blocks(
            q.cuda(), bounds, torch.from_numpy(table)[None].cuda(), torch.tensor([L], **i32),
            torch.tensor([0, 1], **i32), 1, L, K, keep_first=1, keep_last=1,
            selected=out[:2 * K].view(1, 2, K))
        assert pa.pa_get_device_error() == 0
        assert (out[2 * K:] == -77).all()
        for h in range(2):
            sq = np.float32(np.abs(x[h]).max() / np.float32(127))
            code = np.rint(x[h] / sq).astype(np.int64)
            H, Lo = hi[table, h].astype(np.int64), lo[table, h].astype(np.int64)
            # (a code of -128 may stand in a record as well)
            dots = (np.maximum(code, 0) @ H.T + np.minimum(code, 0) @ Lo.T).max(0)
            with np.errstate(all="ignore"):
                score = _order(dots.astype(np.float32) * sc[table, h])
            mid = sorted(range(1, n - 1), key=lambda b: (-score[b], b))[:K - 2]
            assert sel[0, h].tolist() == sorted([0, n - 1] + mid)


@pytest.mark.parametrize("T", [3, 20])
def test_lists_do_not_depend_on_the_longest_length_named(T):
    """max_seq_len chooses how a row's keys are held (registers of 256 or 1024
    threads, or read again); 24 rows and 160 of them, the same lists."""
    lens = [(15000 - 100 * i, 1) for i in range(T)]
    wl, md, dev = step(lens, 16, 8, 64)
    bounds = _random_bounds(wl.k_cache.shape[0], 8, 64, T, ties=True)
    hi, lo, sc = ref.records(bounds, 64)
    want = ref.select(wl.q.float().numpy(), hi, lo, sc, md, 2, 40, 1, 2)
    for blocks in (938, 1024, 1025, 4096, 4097, 8192, 8193, 16384, 16385, 20001):
        table = torch.zeros(T, blocks, dtype=torch.int32, device="cuda")
        table[:, :938] = dev["block_tables"][:, :938]
        sel, cnt = pa.pa_select_blocks(wl.q.cuda(), bounds, table, dev["seq_lens"],
                                       dev["query_start_loc"], 1, 16 * blocks, 40, 1, 2)
        assert pa.pa_get_device_error() == 0
        sel = sel.cpu()
        for (t, h), b in want.items():
            assert sel[t, h].tolist() == b, (blocks, t, h)


def test_passes_over_the_step_do_not_change_the_result():
    """A step whose scores exceed the workspace's bound runs in passes."""
    lens = [(16384, 64)] * 4 + [(20000, 1)] * 3
    wl, md, dev = step(lens, 8, 8, 64)
    bounds = _random_bounds(wl.k_cache.shape[0], 8, 64, 9)
    # max_seq_len raised so that the 259 tokens need three passes
    T = wl.num_tokens
    big = 16 * ((48 << 20) // (8 * 4 * 100))
    wide = torch.zeros(len(lens), big // 16, dtype=torch.int32, device="cuda")
    wide[:, :dev["block_tables"].shape[1]] = dev["block_tables"]
    assert pa.pa_select_blocks_workspace_size(T, 8, big) < T * 8 * 4 * (big // 16)
    a = pa.pa_select_blocks(wl.q.cuda(), bounds, *meta(dev), 64, 20000, 40)
    b = pa.pa_select_blocks(wl.q.cuda(), bounds, wide, dev["seq_lens"],
                            dev["query_start_loc"], 64, big, 40)
    assert pa.pa_get_device_error() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_of_no_request_are_left_and_bad_metadata_is_flagged():
    wl, md, dev = step([(700, 2), (90, 1)], 4, 2, 64)
    bounds = _random_bounds(wl.k_cache.shape[0], 2, 64, 5)
    q = torch.cat([wl.q, wl.q]).cuda()  # three rows of no request
    sel = torch.full((6, 2, 4), -77, dtype=torch.int32, device="cuda")
    cnt = torch.full((6, 2), -77, dtype=torch.int32, device="cuda")
    _select(wl, dev, md, bounds, 4, 1, 1, q=q, selected=sel, num_selected=cnt)
    assert pa.pa_get_device_error() == 0
    assert (sel[3:] == -77).all() and (cnt[3:] == -77).all() and (cnt[:3] == 4).all()
    # lengths beyond max_seq_len: flagged, rows left
    sel.fill_(-77)
    pa.pa_select_blocks(q, bounds, *meta(dev), 2, 600, 4, selected=sel, num_selected=cnt)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
    assert (sel[:2] == -77).all() and (sel[2, :, 0] == 0).all()
    # a block id out of range: flagged, never read
    bad = dev["block_tables"].clone()
    bad[0, 5], bad[0, 6] = -4, 1 << 30
    pa.pa_select_blocks(q, bounds, bad, dev["seq_lens"], dev["query_start_loc"], 2, 700, 4,
                        selected=sel, num_selected=cnt)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_BLOCK_ID
    rec = bounds.clone()
    bad[1, 5] = 1 << 30
    pa.pa_summarise_blocks(wl.k_cache.cuda(), rec, bad, dev["seq_lens"],
                           dev["query_start_loc"], 3, 2, 700)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_BLOCK_ID
    pa.pa_summarise_blocks(wl.k_cache.cuda(), rec, dev["block_tables"], dev["seq_lens"],
                           dev["query_start_loc"], 3, 1, 700)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
