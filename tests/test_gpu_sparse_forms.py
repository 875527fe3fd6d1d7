"""Every form that the sparse decode step's kernels are built in: each pair of
types, head dim and number of heads, and steps of many tokens."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref
from tests.test_gpu_attention_selected import PROB, _lists, _run
from tests.test_gpu_norm_rope import _bits, _cache, _check_rows, _inputs, _table, _weights
from tests.test_gpu_select import meta, step
from tests.test_gpu_sparse_edges import _attend

pytestmark = pytest.mark.gpu


FORMS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3"),
         ("bf16", "int4"), ("f16", "int4"), ("bf16", "nvfp4"), ("f16", "nvfp4")]


@pytest.mark.parametrize("group", [1, 7, 9, 16, 17])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,cache", FORMS)
def test_every_form_of_selected_attention(dtype, cache, D, group):
    """Head counts on both sides of eight and sixteen, over every pair of types:
    ragged lists, empty ones and long ones that the shares cut."""
    wl, md, dev = step([(5000, 2), (3, 1), (16, 1), (333, 9), (1000, 1)], 2 * group, 2, D, dtype,
                       cache)
    lists = _lists(np.random.default_rng(group), md, 2, 300, "ragged")
    lists[0, 0] = list(range(300))
    out = _run(wl, md, dev, lists, 300)
    assert pa.pa_get_device_error() == 0
    want, mag, qk = _attend(wl, md, lists)
    tol = ref.attend_tolerance(want, mag, qk, dtype, PROB[cache])
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("group", [1, 4, 5, 8, 9, 20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_form_of_the_selection(dtype, D, group):
    """Groups on both sides of four heads (columns twice) and of eight (passes
    over the records), with eleven KV heads (two CTAs' worth)."""
    wl, md, dev = step([(3000, 2), (90, 1), (1500, 1)], 11 * group, 11, D, dtype)
    bounds = _any_bounds(wl.k_cache.shape[0], 11, D, group)
    sel, cnt = pa.pa_select_blocks(wl.q.cuda(), bounds, *meta(dev), md["max_query_len"],
                                   md["max_seq_len"], 30, keep_first=2, keep_last=3)
    assert pa.pa_get_device_error() == 0
    want = ref.select(wl.q.float().numpy(), *ref.records(bounds, D), md, group, 30, 2, 3)
    sel, cnt = sel.cpu().numpy(), cnt.cpu().numpy()
    for (t, h), blocks in want.items():
        assert cnt[t, h] == len(blocks)
        np.testing.assert_array_equal(sel[t, h], blocks + [-1] * (30 - len(blocks)))


def _any_bounds(NB, H, D, seed):
    rng = np.random.default_rng(seed)
    b = np.zeros((NB, H, pa.bounds_bytes(D)), dtype=np.uint8)
    hi = rng.integers(-127, 128, (NB, H, D))
    b[..., :D] = hi.astype(np.int8).view(np.uint8)
    b[..., D:2 * D] = np.minimum(hi, rng.integers(-127, 128, (NB, H, D))).astype(
        np.int8).view(np.uint8)
    b[..., 2 * D:2 * D + 4] = rng.uniform(0, 0.05, (NB, H, 1)).astype(np.float32).view(np.uint8)
    return torch.from_numpy(b).cuda()


@pytest.mark.parametrize("H", [1, 7, 8, 9, 20])
@pytest.mark.parametrize("cache", ["f32", "f16", "bf16", "e4m3", "int4", "nvfp4"])
def test_summaries_of_any_number_of_heads(cache, H):
    """A warp to each KV head, eight to a CTA."""
    for D in (64, 128):
        wl, md, dev = step([(70, 30), (16, 1), (9, 9)], H, H, D,
                           cache if cache in ("f32", "f16") else "bf16", cache)
        got = torch.full((wl.k_cache.shape[0], H, pa.bounds_bytes(D)), 0xA5, dtype=torch.uint8,
                         device="cuda")
        pa.pa_summarise_blocks(wl.k_cache.cuda(), got, *meta(dev), wl.num_tokens,
                               md["max_query_len"], md["max_seq_len"], cache_dtype=cache)
        assert pa.pa_get_device_error() == 0
        k = ref.decode_pages(wl.k_cache, cache, D)
        hi, lo, s = ref.records(got, D)
        left = np.ones(len(k), dtype=bool)
        for r, (L, n) in enumerate([(70, 30), (16, 1), (9, 9)]):
            for b in range((L - n) // 16, -(-L // 16)):
                blk = md["block_tables"][r, b]
                left[blk] = False
                for h in range(H):
                    w = ref.bounds_of(k[blk, h, :min(16, L - 16 * b)])
                    np.testing.assert_array_equal(hi[blk, h], w[0])
                    np.testing.assert_array_equal(lo[blk, h], w[1])
                    assert s[blk, h] == w[2]
        assert (got[torch.from_numpy(left).cuda()] == 0xA5).all()


LARGE = [("bf16", "bf16", 128, False), ("bf16", "bf16", 64, True), ("f16", "f16", 128, True),
         ("f32", "f32", 128, False), ("f32", "f32", 64, True), ("bf16", "e4m3", 128, True),
         ("bf16", "e4m3", 64, False), ("f32", "e4m3", 128, False), ("bf16", "int4", 128, False),
         ("f16", "int4", 64, True), ("f32", "int4", 128, True), ("bf16", "nvfp4", 128, False),
         ("f16", "nvfp4", 64, True), ("f32", "nvfp4", 128, False), ("bf16", "nvfp4", 128, True)]


@pytest.mark.parametrize("rot", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("dtype,cache,D,inter", LARGE)
def test_rotations_of_steps_that_take_several_rows_a_lane(dtype, cache, D, inter, rot):
    """Steps large enough for eight heads per lane group, with head counts that
    fill no group: the formula's queries and keys, and the cached bits of
    pa_reshape_and_cache on them."""
    Hq, Hkv = 37, 5
    T = 900 if D == 128 else 1750  # x 47 rows: past 16 warps of 8 x 2 (4) rows on 152 SMs
    i = _inputs(D + len(cache), T, Hq, Hkv, D, dtype)
    i["k"][5], i["v"][6] = 0, 0
    qw, kw, qwn, kwn = _weights(i, "same", dtype)
    R = int(D * rot)
    cs = _table(700, R) if R else None
    turn = (torch.from_numpy(i["pos"]).cuda(), torch.from_numpy(cs).cuda()) if R else (None, None)
    slots = torch.from_numpy(i["slots"]).cuda()
    same = [_cache(i["nb"], Hkv, D, dtype, i["rng"]) for _ in range(2)]
    out = pa.pa_norm_rope_and_cache(i["q"], i["k"], i["v"], *same, slots, *turn, qw, kw,
                                    interleaved=inter)
    _check_rows(out, i["q"], qwn, 1e-6, cs, i["pos"], inter, dtype)
    keys = same[0][i["slots"] // 16, :, i["slots"] % 16].contiguous()
    _check_rows(keys, i["k"], kwn, 1e-6, cs, i["pos"], inter, dtype)
    if cache == dtype:
        b, o = i["slots"] // 16, i["slots"] % 16
        assert torch.equal(_bits(same[1][b, :, o]), _bits(i["v"].contiguous()))
    else:
        init = [_cache(i["nb"], Hkv, D, cache, i["rng"]) for _ in range(2)]
        got, want = [t.clone() for t in init], [t.clone() for t in init]
        sc = dict(k_scale=0.37, v_scale=0.011, cache_dtype=cache)
        out2 = pa.pa_norm_rope_and_cache(i["q"], i["k"], i["v"], *got, slots, *turn, qw, kw,
                                         interleaved=inter, **sc)
        pa.pa_reshape_and_cache(keys, i["v"], *want, slots, **sc)
        assert torch.equal(_bits(out), _bits(out2))
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert pa.pa_get_device_error() == 0
