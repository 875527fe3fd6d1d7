"""The sparse decode step's operators at their edges: the sizes, values and
streams where a result could be wrong although the ordinary cases are right."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref
from tests.test_gpu_attention_selected import PROB, _lists, _run, _tensors
from tests.test_gpu_select import meta, step
from tests.test_gpu_sparse_step import Loop

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _summarise_whole(kc, blocks, H, D, cache):
    """Records of `blocks` full blocks of one request."""
    got = torch.zeros(blocks, H, pa.bounds_bytes(D), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 16 * blocks
    pa.pa_summarise_blocks(kc, got, torch.arange(blocks, **i32)[None].contiguous(),
                           torch.tensor([n], **i32), torch.tensor([0, n], **i32), n, n, n,
                           cache_dtype=cache)
    assert pa.pa_get_device_error() == 0
    return ref.records(got, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["f32", "int4"])
def test_codes_of_subnormal_keys(cache, D):
    """Keys of a few units of 2^-149: the scale is a subnormal of few bits, and
    quotients go past 127 on either side.  Codes stay in [-127, 127]."""
    rng = np.random.default_rng(D)
    unit = np.array([-130, 178, -178, 190, -190, -127, 1000, -1000, 65, 1, -1, -5000])
    B = len(unit)
    if cache == "f32":
        keys = np.broadcast_to(unit[:, None, None].astype(np.float64), (B, 16, D)) * 2.0 ** -149
        keys = keys.copy()
        keys[-1] *= rng.integers(1, 4, (16, D))
        kc = torch.from_numpy(keys.astype(np.float32)).view(B, 1, 16, D).cuda()
    else:  # codes of one sign, scales of a few units
        page = np.zeros((B, 1, pa.page_bytes_4bit("int4", D)), dtype=np.uint8)
        for b in range(B):
            code = int(np.sign(unit[b])) * (rng.integers(1, 8, (16, D)) if b % 3 == 2 else
                                            np.ones((16, D), dtype=np.int64))
            nib = (code & 15).astype(np.uint8)
            page[b, 0, :8 * D] = (nib[:, ::2] | nib[:, 1::2] << 4).reshape(-1)
            sc = np.full(16, abs(int(unit[b])), np.uint32)  # the bits of units of 2^-149
            page[b, 0, 8 * D:] = sc.view(np.uint8)
        kc = torch.from_numpy(page).cuda()
        keys = ref.decode_pages(kc, "int4", D)[:, 0]
    hi, lo, s = _summarise_whole(kc, B, 1, D, cache)
    for b in range(B):
        w = ref.bounds_of(keys[b])
        np.testing.assert_array_equal(hi[b, 0], w[0])
        np.testing.assert_array_equal(lo[b, 0], w[1])
        assert s[b, 0] == w[2]


def _attend(wl, md, lists, scale=None):
    D, c = wl.head_dim, wl.cache_dtype
    scaled = c in ("e4m3", "nvfp4")
    return ref.attend(
        wl.q.double().numpy(), ref.decode_pages(wl.k_cache, c, D),
        ref.decode_pages(wl.v_cache, c, D), md, lists, wl.group,
        wl.scale if scale is None else scale, wl.k_scale if scaled else 1.0,
        wl.v_scale if scaled else 1.0)


@pytest.mark.parametrize("blocks", [1, 3, 29, 2000])
@pytest.mark.parametrize("dtype,group", [("bf16", 4), ("bf16", 16), ("f16", 4), ("f32", 4),
                                         ("f32", 8)])
def test_an_infinite_value_makes_its_channel_infinite(dtype, group, blocks):
    """Wherever in the list it stands, and whether or not the shares cut the list
    (2000 blocks: some 250 parts, no multiple of those that the join loads at a
    time); two infinities of both signs make NaN."""
    wl, md, dev = step([(16 * blocks, 1)], group, 1, 128, dtype)
    lists = {(0, 0): list(range(blocks))}
    at = md["block_tables"][0]
    inf = float("inf")
    wl.v_cache[at[0], 0, 3, 8] = inf
    wl.v_cache[at[blocks - 1], 0, 15, 5] = inf
    wl.v_cache[at[blocks - 1], 0, 7, 77] = -inf
    wl.v_cache[at[blocks // 2], 0, 9, 101] = inf
    wl.v_cache[at[blocks - 1], 0, 0, 101] = -inf
    # scores so near that no probability vanishes in the product's type
    out = _run(wl, md, dev, lists, blocks, scale=0.01).cpu()
    assert pa.pa_get_device_error() == 0
    assert (out[..., 5] == inf).all() and (out[..., 8] == inf).all()
    assert (out[..., 77] == -inf).all() and out[..., 101].isnan().all()
    rest = torch.ones(128, dtype=torch.bool)
    rest[[5, 8, 77, 101]] = False
    wl.v_cache[..., ~rest] = 0
    want, mag, qk = _attend(wl, md, lists, 0.01)
    tol = ref.attend_tolerance(want, mag, qk, dtype, PROB[dtype])
    err = np.abs(out.double().numpy() - want)
    assert (err <= tol)[..., rest.numpy()].all()


@pytest.mark.parametrize("blocks", [2, 2000])
@pytest.mark.parametrize("cache", ["bf16", "f16", "f32", "e4m3", "int4", "nvfp4"])
def test_a_nan_query_makes_its_head_nan(cache, blocks):
    """All of a head's scores are NaN, in every warp and every part."""
    dtype = cache if cache in ("f16", "f32") else "bf16"
    wl, md, dev = step([(16 * blocks - 3, 1)], 4, 1, 128, dtype, cache)
    wl.q[0, 2, 17] = float("nan")
    lists = {(0, 0): list(range(blocks))}
    out = _run(wl, md, dev, lists, blocks).cpu()
    assert pa.pa_get_device_error() == 0
    assert out[0, 2].isnan().all() and out[0, [0, 1, 3]].isfinite().all()


@pytest.mark.parametrize("blocks", [1, 2, 5, 2000])
@pytest.mark.parametrize("cache", ["bf16", "f16", "f32", "e4m3"])
def test_a_nan_key_alone_in_its_block(cache, blocks):
    """The token's own key is the only visible one of the last block: its NaN is
    the only score of the warp that takes the block."""
    dtype = cache if cache in ("f16", "f32") else "bf16"
    wl, md, dev = step([(16 * blocks - 15, 1)] * 2, 8, 2, 128, dtype, cache)
    last = int(md["block_tables"][0, blocks - 1])
    wl.k_cache[last, 1, 0, 3] = 0x7F if cache == "e4m3" else float("nan")
    lists = {(t, h): list(range(blocks)) for t in range(2) for h in range(2)}
    out = _run(wl, md, dev, lists, blocks).cpu()
    assert pa.pa_get_device_error() == 0
    assert out[0, 4:].isnan().all() and out[0, :4].isfinite().all()
    assert out[1].isfinite().all()


@pytest.mark.parametrize("group,D", [(4, 128), (8, 64), (16, 128), (20, 64)])
def test_probabilities_over_bf16_pages_keep_16_bits(group, D):
    """Lists of few keys, whose values nearly cancel: what is left shows the
    probabilities' own rounding.  Each is a head of 8 significant bits, cut off
    (the tail is less than 2^-7 of it), and the tail rounded to 8 bits: off by at
    most 2^-16 of the probability, and so 2^-16 of sum p |v|.  The fp32
    arithmetic is as in attend_tolerance."""
    lens = [(L, 1) for L in (1, 2, 3, 5, 16, 17, 31, 48)] + [(7, 7)]
    wl, md, dev = step(lens, 2 * group, 2, D)
    sign = torch.tensor([1.0, -1.0] * 8)[None, None, :, None]
    wl.v_cache = (wl.v_cache.float() * 0.125 + 8 * sign).bfloat16()
    lists = _lists(None, md, 2, 3, "all")
    out = _run(wl, md, dev, lists, 3)
    assert pa.pa_get_device_error() == 0
    want, mag, qk = _attend(wl, md, lists)
    tol = (ref.half("bf16") * np.abs(want) + (1 + ref.half("bf16")) * (
        2.0 ** -16 * mag + 2.0 ** -16 * (1 + qk) * mag + 2.0 ** -24))
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


def test_short_lists_are_within_the_bar_of_pa_attention():
    """N(0, 1) keys and values, lists of 1 to 48 keys: 2e-3 and half a step of
    the output, and pa_attention, which is within the same, no further off."""
    lens = [(1 + i % 48, 1) for i in range(144)]
    wl, md, dev = step(lens, 32, 8, 128)
    lists = _lists(None, md, 8, 3, "all")
    out = _run(wl, md, dev, lists, 3).double().cpu().numpy()
    full = pa.pa_attention(wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda(), *meta(dev),
                           md["max_query_len"], md["max_seq_len"], wl.scale)
    assert pa.pa_get_device_error() == 0
    want, _, _ = _attend(wl, md, lists)
    bar = 2e-3 + ref.half("bf16") * np.abs(want)
    assert (np.abs(out - want) <= bar).all()
    assert (np.abs(full.double().cpu().numpy() - want) <= bar).all()


@pytest.mark.parametrize("D", [64, 128])
def test_int4_values_with_scales_of_either_sign(D):
    """The values' scales go into the probabilities, whose two parts have their
    sign: pages that another writer left with negative scales are read as such."""
    wl, md, dev = step([(200, 1), (77, 2), (1, 1)], 16, 2, D, "bf16", "int4")
    scales = wl.v_cache[..., 8 * D:].contiguous().view(torch.float32)
    scales[..., 1::2] *= -1
    wl.v_cache[..., 8 * D:] = scales.view(torch.uint8)
    lists = _lists(np.random.default_rng(8), md, 2, 8)
    out = _run(wl, md, dev, lists, 8)
    assert pa.pa_get_device_error() == 0
    want, mag, qk = _attend(wl, md, lists)
    # two parts of a probability times its scale: off by 2^-16, as over bf16 pages
    tol = (ref.half("bf16") * np.abs(want) + (1 + ref.half("bf16")) * (
        2.0 ** -16 * mag + 2.0 ** -16 * (1 + qk) * mag + 2.0 ** -24))
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("size", [1e5, 1e9, 1e13, 1e30])
@pytest.mark.parametrize("cache", ["bf16", "f16", "f32", "e4m3", "int4", "nvfp4"])
def test_scores_far_past_the_exponentials_range(cache, size):
    """Finite scores of any size: a row whose largest score leads by more than
    the scores' rounding is that key's value, and none is NaN."""
    dtype = cache if cache in ("f16", "f32") else "bf16"
    wl, md, dev = step([(200, 1), (77, 2), (1, 1), (16, 1)], 16, 2, 128, dtype, cache)
    lists = _lists(np.random.default_rng(6), md, 2, 8)
    out = _run(wl, md, dev, lists, 8, scale=size).double().cpu().numpy()
    assert pa.pa_get_device_error() == 0
    assert np.isfinite(out).all()
    k, v = (ref.decode_pages(c, cache, 128) for c in (wl.k_cache, wl.v_cache))
    v = v * (wl.v_scale if cache in ("e4m3", "nvfp4") else 1.0)
    sure = 0
    for t, r, p in ref.tokens_of(md):
        for h in range(2):
            keys = [j for b in lists[t, h] for j in range(16 * b, min(16 * b + 16, p + 1))]
            at = md["block_tables"][r, np.array(keys) // 16], h, np.array(keys) % 16
            for g in range(8 * h, 8 * h + 8):
                x = wl.q[t, g].double().numpy()
                score = k[at] @ x
                best = int(score.argmax())
                # (fp32 sums of 128 products: 2^-17 of the terms' sum covers them)
                lead = score[best] - np.partition(score, -2)[-2] if len(score) > 1 else np.inf
                slack = 2.0 ** -16 * (np.abs(k[at]) @ np.abs(x)).max()
                # and 2^-40 of the others' weight, at the smallest of the scales
                if lead > slack + 40 / size:
                    sure += 1
                    want = v[at][best]
                    assert (np.abs(out[t, g] - want) <= ref.half(dtype) * np.abs(want) +
                            2.0 ** -20).all()
    assert sure >= 60


@pytest.mark.parametrize("cache,D", [("e4m3", 128), ("e4m3", 64), ("int4", 128), ("int4", 64),
                                     ("nvfp4", 128), ("nvfp4", 64)])
@pytest.mark.parametrize("power", [-100, -40, -12, 0])
def test_small_queries_over_narrow_pages(cache, D, power):
    """The products are in f16, the bf16 queries reach far below its range: a
    query times 2^power and a scale divided by it give the same scores."""
    wl, md, dev = step([(200, 1), (77, 2), (16, 1)], 16, 2, D, "bf16", cache)
    scale = wl.scale * 2.0 ** -power
    wl.q *= 2.0 ** power
    lists = _lists(np.random.default_rng(3), md, 2, 8)
    out = _run(wl, md, dev, lists, 8, scale=scale)
    assert pa.pa_get_device_error() == 0
    want, mag, qk = _attend(wl, md, lists, scale)
    tol = ref.attend_tolerance(want, mag, qk, "bf16", "f16")
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("group", [4, 8, 12])
@pytest.mark.parametrize("cache", ["e4m3", "int4", "nvfp4"])
def test_heads_of_very_different_sizes_over_narrow_pages(cache, group):
    """Each head is brought into f16's range by a power of two of its own: a
    head beside one 2^40 times as large keeps its bits."""
    wl, md, dev = step([(200, 1), (77, 2), (16, 1)], 2 * group, 2, 128, "bf16", cache)
    wl.q[:, 1::3] *= 2.0 ** 40
    wl.q[:, 2::5] *= 2.0 ** -30
    lists = _lists(np.random.default_rng(4), md, 2, 8)
    out = _run(wl, md, dev, lists, 8)
    assert pa.pa_get_device_error() == 0
    want, mag, qk = _attend(wl, md, lists)
    tol = ref.attend_tolerance(want, mag, qk, "bf16", "f16")
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_one_token_of_a_qkv_row_in_place():
    """A single token's slice of a QKV row is contiguous whatever its row
    stride: its rotation in place is the one into a buffer."""
    Hq, Hkv, D = 8, 2, 128
    g = torch.Generator("cuda").manual_seed(5)
    qkv = torch.randn(1, (Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv.view(1, Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), dim=1)
    assert q.is_contiguous() and q.stride(0) != Hq * D
    cs = torch.randn(9, D, generator=g, device="cuda")
    pos = torch.tensor([7], dtype=torch.int32, device="cuda")
    slot = torch.tensor([21], device="cuda")
    w = torch.rand(D, generator=g, device="cuda").bfloat16()
    kc, vc = (torch.zeros(2, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    want = pa.pa_norm_rope_and_cache(q, k, v, kc, vc, slot, pos, cs, w, w)
    keys = kc.clone(), vc.clone()
    kc.zero_(), vc.zero_()
    rest = qkv[:, Hq * D:].clone()
    got = pa.pa_norm_rope_and_cache(q, k, v, kc, vc, slot, pos, cs, w, w, q_out=q)
    assert pa.pa_get_device_error() == 0
    assert got is q and torch.equal(q, want) and torch.equal(qkv[:, Hq * D:], rest)
    assert torch.equal(kc, keys[0]) and torch.equal(vc, keys[1])


class Spy:
    """The library, with the arguments of the last call."""

    def __init__(self, lib):
        self.lib, self.args = lib, None

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            if not name.endswith("_size"):
                self.args = args
            return f(*args)
        return call


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", ["select", "selected", "attention", "window", "cascade"])
def test_a_workspace_belongs_to_the_stream_it_is_used_on(name, as_handle, monkeypatch):
    """A call on another stream than the current one: what it allocates is not
    handed out again on the current stream while the kernels may still use it."""
    wl, md, dev = step([(900, 1), (64, 1)], 8, 2, 128)
    q, kc, vc = wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda()
    lists = {(t, h): [0, 2, 3] for t in range(2) for h in range(2)}
    sel, cnt = _tensors(lists, 2, 2, 3)
    bounds = torch.ones(kc.shape[0], 2, pa.bounds_bytes(128), dtype=torch.uint8, device="cuda")
    table = dev["block_tables"].clone()
    table[:, 0] = table[0, 0]
    m = (dev["seq_lens"], dev["query_start_loc"])
    run = {
        "select": lambda s: pa.pa_select_blocks(q, bounds, table, *m, 1, 900, 3, stream=s)[0],
        "selected": lambda s: pa.pa_attention_selected(q, kc, vc, table, *m, 1, 900, wl.scale,
                                                       sel, cnt, stream=s),
        "attention": lambda s: pa.pa_attention(q, kc, vc, table, *m, 1, 900, wl.scale,
                                               stream=s),
        "window": lambda s: pa.pa_attention_window(q, kc, vc, table, *m, 1, 900, wl.scale, 100,
                                                   stream=s),
        "cascade": lambda s: pa.pa_attention_cascade(q, kc, vc, table, *m, 1, 900, wl.scale, 1,
                                                     stream=s)}[name]
    want = run(None)
    spy = Spy(pa.load_library())
    monkeypatch.setattr(pa, "_lib", spy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(side.cuda_stream if as_handle else side)
    ws, nbytes, handle = spy.args[-3:]
    assert handle == side.cuda_stream and nbytes > 0
    again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")  # (not written)
    assert again.data_ptr() + nbytes <= ws or ws + nbytes <= again.data_ptr()
    side.synchronize()
    assert torch.equal(got, want) and pa.pa_get_device_error() == 0


BUILD_SIZES = """
import sys
import numpy as np
import torch
from tests.test_gpu_build_step import _case, _run
# ascending: no earlier call has raised the kernel's shared memory
for B in (4071, 4072, 4073, 4096, 4097, 16384, 4096, 64):
    rng = np.random.default_rng(B)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, 40, B), rng.integers(0, 3, B))]
    _run(_case(rng, lens, pad=3))
print("sizes ok")
"""


def test_step_sizes_around_48_kb_of_shared_memory():
    """The kernel's static shared memory counts too: a fresh process, since the
    opt-in to more lasts for the process."""
    r = subprocess.run([sys.executable, "-c", BUILD_SIZES], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "sizes ok" in r.stdout, r.stderr[-2000:]


def test_steps_of_different_sizes_from_two_threads():
    """Each thread's launches find the shared memory that they need, whatever the
    other asks for between."""
    failed = []

    def loop(B):
        try:
            i32 = dict(dtype=torch.int32, device="cuda")
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                new, done = torch.ones(B, **i32), torch.zeros(B, **i32)
                table = torch.full((B, 1), -1, **i32)
                free, count = torch.arange(B, **i32), torch.tensor([B], **i32)
                for _ in range(300):
                    out = pa.pa_build_step(new, done, table, free, count, B, B)
                stream.synchronize()
                assert int(out[4]) == 0 and out[1][-1] == B
                assert torch.equal(out[3], 16 * torch.arange(B - 1, -1, -1, device="cuda"))
        except Exception as e:  # noqa: BLE001 (a thread's failure is the test's)
            failed.append((B, e))

    threads = [threading.Thread(target=loop, args=(B,)) for B in (16384, 4200, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("op", ["summarise", "select", "selected", "attention"])
@pytest.mark.parametrize("broken", ["length", "offset", "last", "table"])
def test_a_broken_request_without_tokens_is_flagged(op, broken):
    """As in pa_attention: every request's metadata is checked, whether or not
    a token points to it, and the other requests' results stand."""
    wl, md, dev = step([(300, 1), (64, 0), (90, 1)], 8, 2, 128)
    q, kc, vc = wl.q.cuda(), wl.k_cache.cuda(), wl.v_cache.cuda()
    L, qsl = dev["seq_lens"].clone(), dev["query_start_loc"].clone()
    rows = [0, 1]
    if broken == "length":
        L[1] = -5
    elif broken == "table":
        L[1] = 16 * dev["block_tables"].shape[1] + 1
    elif broken == "offset":
        qsl[2] = 0  # requests 1 and 2: of -1 tokens, and of two
        rows = [0]
    else:
        qsl[3] = -1
        rows = [0]
    lists = {(t, h): [0, 2, 3] for t in range(2) for h in range(2)}
    sel, cnt = _tensors(lists, 2, 2, 3)
    bounds = _bounds(kc, 2)

    def run(L, qsl):
        m = (dev["block_tables"], L, qsl)
        if op == "summarise":
            out = bounds.clone()
            pa.pa_summarise_blocks(kc, out, *m, 2, 1, 300)
            # of each token's own block
            return torch.stack([out[int(md["block_tables"][r, p // 16])]
                                for r, p in ((0, 299), (2, 89))])
        if op == "select":
            return pa.pa_select_blocks(q, bounds, *m, 1, 300, 3)[0]
        if op == "selected":
            return pa.pa_attention_selected(q, kc, vc, *m, 1, 300, wl.scale, sel, cnt)
        return pa.pa_attention(q, kc, vc, *m, 1, 300, wl.scale)

    want = run(dev["seq_lens"], dev["query_start_loc"])
    assert pa.pa_get_device_error() == 0
    got = run(L, qsl)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_METADATA
    got, want = got[rows], want[rows]
    if op == "attention":  # split-K ranges follow the work there is
        assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * (1 + want.abs())).all()
    else:
        assert torch.equal(got, want)


def _bounds(kc, Hkv):
    rng = np.random.default_rng(9)
    b = rng.integers(0, 100, (kc.shape[0], Hkv, pa.bounds_bytes(128)), dtype=np.uint8)
    b[..., 256:260] = np.array([0.01], np.float32).view(np.uint8)
    return torch.from_numpy(b).cuda()


def test_the_step_ends_at_the_first_request_without_a_block():
    """The requests before it run, it and those behind it wait, one that needs
    no block among them; a released block lets them go on."""
    loop = Loop(11, [16, 40, 32, 30])
    loop.prefill()
    loop.count.fill_(1)
    b = loop.buffers(4)
    loop.fill(b, [1, 1, 1, 1])
    loop.step(b, 1)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_NO_BLOCKS
    assert loop.lens.tolist() == [17, 41, 32, 30] and b["qsl"].tolist() == [0, 1, 2, 2, 2]
    loop.check(b)
    loop.count.fill_(1)
    loop.fill(b, [0, 0, 1, 1])
    loop.step(b, 1)
    assert pa.pa_get_device_error() == 0
    assert loop.lens.tolist() == [17, 41, 33, 31]
    loop.check(b)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_copied_block_gets_its_record_in_the_step_that_writes_to_it(cache):
    """A request forked in the middle of a block: the block is copied, the next
    token goes into the copy, and that step's summary makes the copy's record
    before the selection reads it, whatever stood there."""
    loop = Loop(12, [40, 1, 75], cache)
    loop.check(loop.prefill())
    new = int(loop.free[int(loop.count) - 1])
    loop.count -= 1
    old = int(loop.table[0, 2])
    loop.table[1, :2] = loop.table[0, :2]
    loop.table[1, 2] = new
    loop.lens[1] = 40
    loop.bounds[new] = 255  # codes of -1 and a NaN scale
    pa.pa_copy_blocks(loop.kc, loop.vc, torch.tensor([[old, new]], device="cuda"))
    b = loop.buffers(3)
    for _ in range(10):  # into the next block
        loop.fill(b, [1, 1, 1])
        loop.step(b, 1)
        loop.check(b)
    assert pa.pa_get_device_error() == 0
    assert not torch.equal(loop.bounds[old], loop.bounds[new])


def test_a_copied_full_block_takes_its_record_along():
    """A copy that no token is written to has no record of its own: the caller
    copies the source's, as the caches' pages."""
    loop = Loop(13, [64, 20])
    loop.check(loop.prefill())
    new = int(loop.free[int(loop.count) - 1])
    loop.count -= 1
    old = int(loop.table[0, 1])
    loop.bounds[new] = 255
    pa.pa_copy_blocks(loop.kc, loop.vc, torch.tensor([[old, new]], device="cuda"))
    loop.bounds[new] = loop.bounds[old]
    loop.table[0, 1] = new
    loop.kc[old], loop.vc[old], loop.bounds[old] = 99, 99, 255
    b = loop.buffers(2)
    loop.fill(b, [1, 1])
    loop.step(b, 1)
    loop.check(b)
    assert pa.pa_get_device_error() == 0
