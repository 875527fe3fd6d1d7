"""pa_attention_selected on the GPU against plain softmax attention over the
listed blocks in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref
from tests.test_gpu_select import meta, step

pytestmark = pytest.mark.gpu


def _lists(rng, md, Hkv, K, kind="random"):
    """Ascending block lists per (token, KV head)."""
    out = {}
    for t, r, p in ref.tokens_of(md):
        n = p // 16 + 1
        for h in range(Hkv):
            if kind == "all":
                out[t, h] = list(range(min(n, K)))
                continue
            k = int(rng.integers(0, min(n, K) + 1)) if kind == "ragged" else min(n, K)
            blocks = rng.permutation(n)[:k]
            if k and kind != "ragged":
                blocks[0] = n - 1 if n - 1 not in blocks else blocks[0]
            out[t, h] = sorted(int(b) for b in blocks)
    return out


def _tensors(lists, T, Hkv, K, fill=-1):
    sel = np.full((T, Hkv, K), fill, dtype=np.int32)
    cnt = np.zeros((T, Hkv), dtype=np.int32)
    for (t, h), b in lists.items():
        sel[t, h, :len(b)] = b
        cnt[t, h] = len(b)
    return torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()


def _run(wl, md, dev, lists, K, scale=None, **kw):
    sel, cnt = _tensors(lists, wl.num_tokens, wl.num_kv_heads, K)
    scale = wl.scale if scale is None else scale
    return pa.pa_attention_selected(
        wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda(), *meta(dev), md["max_query_len"],
        md["max_seq_len"], scale, sel, cnt, wl.k_scale, wl.v_scale,
        cache_dtype=wl.cache_dtype, **kw)


PROB = {"bf16": "bf16", "f16": "f16", "f32": "f32", "e4m3": "f16", "int4": "f16",
        "nvfp4": "f16"}


def _check(wl, md, lists, out, scale=None):
    D, c = wl.head_dim, wl.cache_dtype
    scaled = c in ("e4m3", "nvfp4")
    want, mag, qk = ref.attend(
        wl.q.double().numpy(), ref.decode_pages(wl.k_cache, c, D),
        ref.decode_pages(wl.v_cache, c, D), md, lists, wl.group,
        wl.scale if scale is None else scale, wl.k_scale if scaled else 1.0,
        wl.v_scale if scaled else 1.0)
    tol = ref.attend_tolerance(want, mag, qk, wl.q_dtype, PROB[c])
    got = out.float().cpu().double().numpy()
    assert not np.isnan(want).any() and np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())
    return want, tol


RAGGED = [(L, 1) for L in (1, 2, 15, 16, 17, 33, 255, 256, 257, 1500)]
CHUNKS = [(300, 40), (17, 17), (1000, 1), (64, 0), (50, 3)]
CASES = {
    # lens, Hq, Hkv, D, dtype, cache, K
    "bf16_g4": (RAGGED, 32, 8, 128, "bf16", "bf16", 12),
    "bf16_g8_chunks": (CHUNKS, 16, 2, 128, "bf16", "bf16", 9),
    "f16_mha": (RAGGED, 3, 3, 128, "f16", "f16", 40),
    "bf16_g5": (RAGGED, 20, 4, 128, "bf16", "bf16", 17),
    "f16_g16": (RAGGED, 32, 2, 128, "f16", "f16", 33),
    "bf16_g20": (CHUNKS, 20, 1, 128, "bf16", "bf16", 21),
    "bf16_g64_d64": (RAGGED, 64, 1, 64, "bf16", "bf16", 11),
    "f16_g8_d64": (CHUNKS, 64, 8, 64, "f16", "f16", 30),
    "e4m3_g8": (RAGGED, 64, 8, 128, "bf16", "e4m3", 12),
    "e4m3_f16_g2_d64": (CHUNKS, 6, 3, 64, "f16", "e4m3", 19),
    "e4m3_g16": (RAGGED, 16, 1, 128, "bf16", "e4m3", 64),
    "e4m3_g12_d64": (RAGGED, 24, 2, 64, "bf16", "e4m3", 7),
    "f32": (RAGGED, 8, 2, 128, "f32", "f32", 12),
    "f32_d64": (CHUNKS, 8, 2, 64, "f32", "f32", 12),
    "int4": (RAGGED, 8, 2, 128, "bf16", "int4", 12),
    "int4_d64": (CHUNKS, 8, 2, 64, "f16", "int4", 12),
    "nvfp4": (RAGGED, 8, 2, 128, "bf16", "nvfp4", 12),
    "nvfp4_d64": (CHUNKS, 8, 2, 64, "f16", "nvfp4", 12),
    "one_request_long_list": ([(20000, 1)], 8, 2, 128, "bf16", "bf16", 1000),
    "one_block": (RAGGED, 8, 2, 128, "bf16", "bf16", 1),
}


@pytest.mark.parametrize("kind", ["random", "ragged"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_attention_over_lists(name, kind):
    lens, Hq, Hkv, D, dtype, cache, K = CASES[name]
    wl, md, dev = step(lens, Hq, Hkv, D, dtype, cache)
    lists = _lists(np.random.default_rng(len(name)), md, Hkv, K, kind)
    out = _run(wl, md, dev, lists, K)
    assert pa.pa_get_device_error() == 0
    _check(wl, md, lists, out)
    again = _run(wl, md, dev, lists, K)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_all_blocks_is_pa_attention(cache):
    wl, md, dev = step([(700, 1), (33, 2), (16, 1), (250, 30)], 32, 8, 128, "bf16", cache)
    K = 64
    lists = _lists(None, md, 8, K, "all")
    out = _run(wl, md, dev, lists, K)
    want, tol = _check(wl, md, lists, out)
    full = pa.pa_attention(wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda(), *meta(dev),
                           md["max_query_len"], md["max_seq_len"], wl.scale, wl.k_scale,
                           wl.v_scale, cache_dtype=cache)
    assert pa.pa_get_device_error() == 0
    # each is within its own bar of the same values
    bar = {"bf16": 2e-3, "e4m3": 2e-2}[cache] + ref.half("bf16") * np.abs(want) + tol
    assert ((out.float() - full.float()).abs().cpu().numpy() <= bar).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale):
    wl, md, dev = step([(600, 1), (40, 5)], 8, 2, 128, "bf16")
    lists = _lists(np.random.default_rng(1), md, 2, 20)
    out = _run(wl, md, dev, lists, 20, scale=scale)
    _check(wl, md, lists, out, scale=scale)


@pytest.mark.parametrize("big", [1e3, 3e5, 1e30])
def test_large_queries_over_fp8_pages(big):
    """Queries past f16's range: the products are in f16, the queries are not."""
    wl, md, dev = step([(200, 1), (77, 2)], 8, 2, 128, "bf16", "e4m3")
    wl.q *= big
    lists = _lists(np.random.default_rng(2), md, 2, 8)
    out = _run(wl, md, dev, lists, 8, scale=0.1 / big)
    _check(wl, md, lists, out, scale=0.1 / big)


def test_empty_lists_give_zeros_and_rows_of_no_request_are_left():
    wl, md, dev = step([(100, 2), (40, 1)], 8, 2, 128)
    q = torch.cat([wl.q, wl.q]).cuda()
    out = torch.full_like(q, 7.0)
    sel = torch.full((6, 2, 3), -1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    sel[0, 1, 0], cnt[0, 1] = 6, 1
    pa.pa_attention_selected(q, wl.k_cache.cuda(), wl.v_cache.cuda(), *meta(dev), 2, 100,
                             wl.scale, sel, cnt, out=out)
    assert pa.pa_get_device_error() == 0
    assert (out[0, :4] == 0).all() and (out[1:3] == 0).all() and (out[3:] == 7).all()
    assert (out[0, 4:] != 0).any()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32")])
def test_bad_entries_are_skipped_and_flagged(dtype, cache):
    wl, md, dev = step([(160, 1), (90, 1)], 8, 2, 128, dtype, cache)
    good = {(t, h): [1, 3, 4] for t in range(2) for h in range(2)}
    want = _run(wl, md, dev, good, 8)
    for entries in ([1, 3, 3, 4], [1, 3, 2, 4], [1, 3, 4, 99], [1, 3, 4, -2]):
        out = _run(wl, md, dev, {k: entries for k in good}, 8)
        assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
        # the same blocks: only the order of the join may differ
        err = (out.float() - want.float()).abs().max()
        assert err <= 2 * ref.half(dtype) * 8, float(err)
    sel, cnt = _tensors(good, 2, 2, 8)
    args = (wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda())
    for bad in (-1, 9):
        c = cnt.clone()
        c[0, 0] = bad
        out = pa.pa_attention_selected(*args, *meta(dev), 1, 160, wl.scale, sel, c)
        assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
        assert (out[0, :4] == 0).all() and torch.equal(out[1], want[1])
    table = dev["block_tables"].clone()
    table[0, 3] = 1 << 29
    out = pa.pa_attention_selected(*args, table, dev["seq_lens"], dev["query_start_loc"], 1,
                                   160, wl.scale, sel, cnt)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_BLOCK_ID
    _check(wl, md, {k: ([1, 4] if k[0] == 0 else [1, 3, 4]) for k in good}, out)


def test_an_infinite_score_and_nan_in_masked_places():
    """One key of an infinite score in an otherwise ordinary row is NaN or the
    key's value as in IEEE; the slots past each length hold NaN throughout
    (every case here runs over such pages)."""
    wl, md, dev = step([(37, 1)], 2, 1, 128, "f32", "f32")
    wl.k_cache[md["block_tables"][0, 0], 0, 4] = -float("inf")
    wl.q.abs_()  # the score of that key: -inf
    lists = {(0, 0): [0, 1, 2]}
    out = _run(wl, md, dev, lists, 3)
    assert pa.pa_get_device_error() == 0
    assert torch.isfinite(out).all()


def test_page_offsets_past_32_bits():
    """A pool whose last pages lie past 2^32 bytes: their blocks are read."""
    Hkv, D = 8, 128
    NB = (1 << 32) // (Hkv * 16 * D * 2) + 40  # 32 KiB a block
    kc = torch.zeros(NB, Hkv, 16, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[-4:] = torch.randn(4, Hkv, 16, D, device="cuda")
    vc[-4:] = torch.arange(4, device="cuda").view(4, 1, 1, 1) + 1.0
    q = torch.randn(1, 8, D, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(NB - 4, NB, **i32)[None].contiguous()
    for b in range(4):
        sel = torch.full((1, Hkv, 1), b, **i32)
        out = pa.pa_attention_selected(q, kc, vc, table, torch.tensor([64], **i32),
                                       torch.tensor([0, 1], **i32), 1, 64, 0.1, sel,
                                       torch.ones(1, Hkv, **i32))
        # the probabilities' and the output's rounding
        assert ((out.float() - (b + 1)).abs() <= 2 * ref.half("bf16") * (b + 1)).all()
    bounds = torch.zeros(NB, Hkv, pa.bounds_bytes(D), dtype=torch.uint8, device="cuda")
    pa.pa_summarise_blocks(kc, bounds, table, torch.tensor([64], **i32),
                           torch.tensor([0, 64], **i32), 64, 64, 64)
    assert pa.pa_get_device_error() == 0
    assert (bounds[-4:, :, 256:260].view(torch.float32) > 0).all()


F32_CASES = [(1, 128, RAGGED, 12), (3, 64, CHUNKS, 9), (4, 64, RAGGED, 30), (5, 128, CHUNKS, 17),
             (8, 128, RAGGED, 40), (8, 64, CHUNKS, 5), (12, 128, CHUNKS, 8), (20, 64, RAGGED, 6),
             (4, 128, [(20000, 1)], 1000), (8, 128, [(9000, 2), (31, 1)], 500)]


@pytest.mark.parametrize("kind", ["random", "ragged"])
@pytest.mark.parametrize("group,D,lens,K", F32_CASES)
def test_fp32_caches(group, D, lens, K, kind):
    """Heads in fours, eights and several parts; keys of one and of half a row of
    lanes; lists within a CTA's share and across many."""
    Hkv = 3 if group < 8 else 2
    wl, md, dev = step(lens, group * Hkv, Hkv, D, "f32")
    lists = _lists(np.random.default_rng(group + K), md, Hkv, K, kind)
    out = _run(wl, md, dev, lists, K)
    assert pa.pa_get_device_error() == 0
    _check(wl, md, lists, out)
    again = _run(wl, md, dev, lists, K)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("dtype,group", [("bf16", 4), ("f16", 16), ("f32", 3), ("f32", 9)])
def test_long_lists_among_many_short_ones(dtype, group):
    """Rows of one to three blocks, empty rows, and two of hundreds: the shares
    cut the long ones and string the short ones together."""
    lens = [(1 + 37 * i % 60, 1) for i in range(90)]
    lens[40], lens[88] = (9000, 1), (7000, 1)
    wl, md, dev = step(lens, 2 * group, 2, 128, dtype)
    K = 600
    lists = _lists(np.random.default_rng(group), md, 2, K)
    for t in (0, 7, 8, 41, 87):
        lists[t, 0] = []
    out = _run(wl, md, dev, lists, K)
    assert pa.pa_get_device_error() == 0
    _check(wl, md, lists, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nan_key_makes_its_heads_nan(dtype):
    """A NaN key that is visible is no -inf: the rows that read it are NaN, as
    the sum of the formula is, wherever in the list it stands; and a row that
    does not list its block is not touched by it."""
    wl, md, dev = step([(200, 1)] * 3, 4, 2, 128, dtype)
    lists = {(t, h): [0, 4, 8, 12] for t in range(3) for h in range(2)}
    for t, block in enumerate((0, 8, 5)):
        wl.k_cache[md["block_tables"][t, block], 1, 0, 7] = float("nan")
    out = _run(wl, md, dev, lists, 4)
    assert pa.pa_get_device_error() == 0
    nan = out.isnan().all(-1).cpu()
    assert nan.tolist() == [[False, False, True, True]] * 2 + [[False] * 4]
    assert out[~nan.cuda()].isfinite().all()


def test_many_rows_with_and_without_lists():
    """More rows than the joining CTAs have threads' worth of in one look, most of
    them empty, some of broken counts; rows of no request behind them."""
    T, Hkv, pad = 20000, 8, 9
    lens, n = T + 40, T
    blocks = -(-lens // 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    kc = torch.randn(blocks, Hkv, 16, 64, generator=g, device="cuda").bfloat16()
    vc = torch.randn(blocks, Hkv, 16, 64, generator=g, device="cuda").bfloat16()
    q = torch.randn(T + pad, Hkv, 64, generator=g, device="cuda").bfloat16()
    table = torch.randperm(blocks, generator=g, device="cuda").int()[None].contiguous()
    sel = torch.zeros(T + pad, Hkv, 1, **i32)
    cnt = (torch.arange((T + pad) * Hkv, **i32).view(T + pad, Hkv) % 7 == 0).int()
    cnt[T:] = 0
    out = torch.full_like(q, 7)
    args = (table, torch.tensor([lens], **i32), torch.tensor([0, n], **i32), n, lens)
    pa.pa_attention_selected(q, kc, vc, *args, 0.1, sel, cnt, out=out)
    assert pa.pa_get_device_error() == 0
    assert (out[T:] == 7).all()
    assert (out[:T][cnt[:T] == 0] == 0).all()
    # block 0 alone, whose 16 keys every one of these tokens sees
    k0, v0 = (c[table[0, 0].long()].double() for c in (kc, vc))
    x = torch.einsum("thd,hjd->thj", q[:T].double(), k0) * float(np.float32(0.1))
    p = torch.softmax(x, -1)
    want = torch.einsum("thj,hjd->thd", p, v0)
    mag = torch.einsum("thj,hjd->thd", p, v0.abs())
    qk = torch.einsum("thd,hjd->thj", q[:T].double().abs(), k0.abs()).amax(-1, True) * 0.1
    tol = torch.from_numpy(ref.attend_tolerance(
        want.cpu().numpy(), mag.cpu().numpy(), qk.cpu().numpy(), "bf16", "bf16")).cuda()
    on = cnt[:T] == 1
    assert ((out[:T].double() - want).abs() <= tol)[on].all()
    cnt[5, 3], cnt[19000, 1] = 2, -3  # of one entry at most: no list, and a flag
    pa.pa_attention_selected(q, kc, vc, *args, 0.1, sel, cnt, out=out)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
    assert (out[5, 3] == 0).all() and (out[19000, 1] == 0).all()
