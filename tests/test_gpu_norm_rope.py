"""pa_norm_rope_and_cache on the GPU: queries and keys against the formulas in
64 bits, the cached bits against pa_reshape_and_cache on the rounded keys."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _table(span, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(span)[:, None] * freq
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _inputs(seed, T, Hq, Hkv, D, dtype, span=700, pad=8):
    rng = np.random.default_rng(seed)
    width = (Hq + 2 * Hkv) * D + pad
    row = torch.from_numpy(
        (rng.standard_normal((T, width)) * rng.uniform(0.05, 20, (T, 1))).astype(np.float32)
    ).to(DT[dtype]).cuda()
    q = row[:, :Hq * D].unflatten(1, (Hq, D))
    k = row[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = row[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    w = [torch.from_numpy(rng.uniform(-1.5, 1.5, D).astype(np.float32)) for _ in range(2)]
    nb = T // 16 + 3
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    pos = rng.integers(0, span, T).astype(np.int32)
    if T > 2:
        pos[:2] = 0, span - 1
    return dict(rng=rng, q=q, k=k, v=v, w=w, nb=nb, slots=slots, pos=pos)


def _cache(nb, Hkv, D, dtype, rng):
    if dtype in ("int4", "nvfp4"):
        shape = (nb, Hkv, pa.page_bytes_4bit(dtype, D))
    else:
        shape = (nb, Hkv, 16, D)
    if dtype in DT:
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(
            DT[dtype]).cuda()
    return torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).cuda()


def _bits(t):
    return t.cpu().view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def _check_rows(got, x, weight, eps, cs, pos, inter, dtype, rows=None):
    """Rounding: half a step of the type, and the fp32 arithmetic.  With the
    norm, the sum of D squares (D / 8 per lane in turn, then a tree: under 12
    roundings deep), the mean, the root, the quotient and two products are at
    most 2^-24 each, relative; the rotation two products and one sum: 24 x
    2^-24 < 2^-19 of the terms' magnitudes."""
    y, m = ref.norm_rope(x.float().cpu().numpy(), weight, eps, cs, pos, inter)
    tol = ref.half(dtype) * np.abs(y) * (1 + 2 ** -8) + 2.0 ** -19 * m + (
        2.0 ** -25 if dtype == "f16" else 2.0 ** -120)
    err = np.abs(got.float().cpu().double().numpy() - y)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert (err <= tol).all(), float((err / tol).max())


CASES = {
    # T, Hq, Hkv, D, dtype, rot, interleaved, weights ("same" / "f32" / None)
    "decode1": (1, 32, 8, 128, "bf16", 128, False, "same"),
    "neox_f16": (37, 8, 2, 128, "f16", 128, False, "f32"),
    "neox_f32": (21, 5, 1, 128, "f32", 128, False, "f32"),
    "pairs_bf16": (50, 4, 4, 128, "bf16", 128, True, "same"),
    "partial_96": (19, 6, 3, 128, "bf16", 96, False, "same"),
    "partial_16": (19, 6, 3, 128, "f16", 16, False, None),
    "partial_pairs_48": (19, 3, 1, 64, "f32", 48, True, "f32"),
    "d64": (100, 14, 2, 64, "bf16", 64, False, "same"),
    "d64_partial_32": (33, 64, 8, 64, "f16", 32, False, "same"),
    "no_rotation": (40, 8, 4, 128, "bf16", 0, False, "same"),
    "no_norm": (40, 8, 8, 64, "f16", 64, True, None),
    "long": (1500, 3, 1, 128, "bf16", 128, False, "same"),
}


def _weights(i, kind, dtype):
    if kind is None:
        return None, None, None, None
    w = [x.to(DT[dtype] if kind == "same" else torch.float32) for x in i["w"]]
    return (w[0].cuda(), w[1].cuda(), w[0].float().numpy(), w[1].float().numpy())


@pytest.mark.parametrize("name", sorted(CASES))
def test_norm_rotation_and_write(name):
    T, Hq, Hkv, D, dtype, rot, inter, kind = CASES[name]
    i = _inputs(len(name) + T, T, Hq, Hkv, D, dtype)
    qw, kw, qwn, kwn = _weights(i, kind, dtype)
    cs = _table(700, rot) if rot else None
    kc, vc = (_cache(i["nb"], Hkv, D, dtype, i["rng"]) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.from_numpy(i["slots"]).cuda()
    out = pa.pa_norm_rope_and_cache(
        i["q"], i["k"], i["v"], kc, vc, slots,
        torch.from_numpy(i["pos"]).cuda() if rot else None,
        torch.from_numpy(cs).cuda() if rot else None, qw, kw, eps=1e-5, interleaved=inter)
    assert pa.pa_get_device_error() == 0
    _check_rows(out, i["q"], qwn, 1e-5, cs, i["pos"], inter, dtype)
    b, o = i["slots"] // 16, i["slots"] % 16
    got_k = kc[b, :, o]
    _check_rows(got_k, i["k"], kwn, 1e-5, cs, i["pos"], inter, dtype)
    assert torch.equal(_bits(vc[b, :, o]), _bits(i["v"].contiguous()))
    k0[b, :, o], v0[b, :, o] = got_k, i["v"]  # everything else is as it was
    assert torch.equal(_bits(kc), _bits(k0)) and torch.equal(_bits(vc), _bits(v0))


@pytest.mark.parametrize("dtype,cache,D", [
    ("bf16", "e4m3", 128), ("f16", "e4m3", 64), ("f32", "e4m3", 128), ("bf16", "int4", 128),
    ("f16", "int4", 64), ("f32", "int4", 128), ("bf16", "nvfp4", 128), ("f16", "nvfp4", 128),
    ("bf16", "nvfp4", 64), ("bf16", "int4", 64)])
def test_quantised_caches_get_the_two_step_bits(dtype, cache, D):
    T, Hq, Hkv = 53, 4, 3
    i = _inputs(D + len(cache), T, Hq, Hkv, D, dtype)
    i["k"][5] = 0
    i["v"][6] = 0
    qw, kw, _, _ = _weights(i, "same", dtype)
    args = (torch.from_numpy(i["slots"]).cuda(), torch.from_numpy(i["pos"]).cuda(),
            torch.from_numpy(_table(700, D)).cuda(), qw, kw)
    same = [_cache(i["nb"], Hkv, D, dtype, i["rng"]) for _ in range(2)]
    out = pa.pa_norm_rope_and_cache(i["q"], i["k"], i["v"], *same, *args)
    keys = same[0][i["slots"] // 16, :, i["slots"] % 16].contiguous()
    init = [_cache(i["nb"], Hkv, D, cache, i["rng"]) for _ in range(2)]
    got, want = [t.clone() for t in init], [t.clone() for t in init]
    sc = dict(k_scale=0.37, v_scale=0.011, cache_dtype=cache)
    out2 = pa.pa_norm_rope_and_cache(i["q"], i["k"], i["v"], *got, *args, **sc)
    pa.pa_reshape_and_cache(keys, i["v"], *want, args[0], **sc)
    assert pa.pa_get_device_error() == 0
    assert torch.equal(_bits(out), _bits(out2))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("off", [1, 3, 4])
def test_rows_that_start_off_16_bytes(off):
    """Odd strides and starts take the scalar loads, with the same result."""
    T, Hq, Hkv, D = 9, 3, 2, 128
    i = _inputs(off, T, Hq, Hkv, D, "bf16", pad=0)
    qw, kw, _, _ = _weights(i, "same", "bf16")
    args = (torch.from_numpy(i["slots"]).cuda(), torch.from_numpy(i["pos"]).cuda(),
            torch.from_numpy(_table(700, D)).cuda(), qw, kw)
    res = []
    for shift in (0, off):
        wide = torch.zeros(T, (Hq + 2 * Hkv) * D + 2 * off, dtype=torch.bfloat16, device="cuda")
        part = wide[:, shift:shift + (Hq + 2 * Hkv) * D] if shift else torch.empty(
            T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
        part[:, :Hq * D] = i["q"].flatten(1)
        part[:, Hq * D:(Hq + Hkv) * D] = i["k"].flatten(1)
        part[:, (Hq + Hkv) * D:] = i["v"].flatten(1)
        kc = torch.zeros(i["nb"], Hkv, 16, D, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        out = pa.pa_norm_rope_and_cache(
            part[:, :Hq * D].unflatten(1, (Hq, D)),
            part[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),
            part[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)), kc, vc, *args)
        res.append([_bits(t) for t in (out, kc, vc)])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_in_place_padding_and_bad_slots_and_positions():
    T, Hq, Hkv, D = 40, 8, 2, 128
    i = _inputs(3, T, Hq, Hkv, D, "bf16")
    qw, kw, qwn, _ = _weights(i, "same", "bf16")
    cs = _table(700, D)
    q = i["q"].contiguous()
    q0 = q.clone()
    slots, pos = i["slots"].copy(), i["pos"].copy()
    slots[[3, 39]] = -1              # padding, positions of any value
    pos[3], pos[39] = -77, 1 << 30
    slots[7] = i["nb"] * 16          # past the cache
    pos[9], pos[11] = 700, -1        # past the table
    kc, vc = (_cache(i["nb"], Hkv, D, "bf16", i["rng"]) for _ in range(2))
    k0 = kc.clone()
    out = pa.pa_norm_rope_and_cache(q, i["k"], i["v"], kc, vc, torch.from_numpy(slots).cuda(),
                                    torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
                                    qw, kw, q_out=q)
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_SLOT | pa.PA_DEV_ERR_METADATA
    assert out is q
    skipped = [3, 7, 9, 11, 39]
    rows = [t for t in range(T) if t not in skipped]
    assert torch.equal(_bits(q[skipped]), _bits(q0[skipped]))
    pos[skipped] = 0
    _check_rows(q, q0, qwn, 1e-6, cs, pos, False, "bf16", rows)
    free = np.setdiff1d(np.arange(i["nb"] * 16), slots[rows])
    assert torch.equal(_bits(kc[free // 16, :, free % 16]), _bits(k0[free // 16, :, free % 16]))


def test_zero_rows_and_large_values():
    """A row of zeros stays zero; values whose squares leave fp32's normal
    range still give finite or IEEE results."""
    q = torch.zeros(3, 1, 64, device="cuda")
    q[1] = 1e18
    q[2] = 1e-30
    w = torch.ones(64, device="cuda")
    kc = torch.zeros(1, 1, 16, 64, device="cuda")
    out = pa.pa_norm_rope_and_cache(q, q, q, kc, torch.zeros_like(kc),
                                    torch.arange(3, device="cuda"), q_weight=w, k_weight=w)
    assert torch.equal(out[0], q[0])
    assert torch.allclose(out[1], torch.ones_like(out[1]), rtol=2.0 ** -20)
    assert torch.allclose(out[2], q[2] * 1e3, rtol=2.0 ** -20)
    assert torch.equal(kc[0, 0, :3], out[:, 0])
