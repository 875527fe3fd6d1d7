"""Plain references of the sparse decode step's operators, in loops and 64
bits (whole numbers and fp32 roundings where the definition names them)."""
from __future__ import annotations

import numpy as np
import torch

import oracle

BS = 16
F32 = np.float32


def half(dtype: str) -> float:
    """Half a step of `dtype`, relative to the value."""
    t = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    return torch.finfo(t).eps / 2


def build_step(query_lens, computed_lens, table, free_blocks, free_count, num_tokens,
               num_blocks):
    """The arrays pa_build_step writes, and its flags (by name)."""
    table = table.copy()
    B, M = table.shape
    flags = set()
    if not 0 <= free_count <= len(free_blocks):
        flags.add("metadata")
        free_count = 0
    need_sum = n_sum = popped = 0
    stopped = False
    seq_lens, qsl, pos, slots = [], [0], [], []
    for r in range(B):
        n, c = int(query_lens[r]), int(computed_lens[r])
        if not 0 <= c <= M * BS:
            flags.add("metadata")
            n = c = 0
        elif n < 0 or c + n > M * BS:
            flags.add("metadata")
            n = 0
        have = -(-c // BS)
        need = -(-(c + n) // BS) - have
        need_sum += need
        n_sum += n
        if need_sum > free_count:
            flags.add("blocks")
            stopped = True
        if n_sum > num_tokens:
            flags.add("metadata")
            stopped = True
        if stopped:
            n = need = 0
        for j in range(need):
            table[r, have + j] = free_blocks[free_count - 1 - popped]
            popped += 1
        for i in range(n):
            p = c + i
            b = int(table[r, p // BS])
            pos.append(p)
            if 0 <= b < num_blocks:
                slots.append(b * BS + p % BS)
            else:
                flags.add("block id")
                slots.append(-1)
        seq_lens.append(c + n)
        qsl.append(qsl[-1] + n)
    pad = num_tokens - len(pos)
    return dict(seq_lens=np.array(seq_lens, dtype=np.int32),
                query_start_loc=np.array(qsl, dtype=np.int32),
                positions=np.array(pos + [0] * pad, dtype=np.int32),
                slot_mapping=np.array(slots + [-1] * pad, dtype=np.int64),
                table=table, free_count=free_count - popped, flags=flags)


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """(y, m): the rotated rows of x [T, H, D] in 64 bits, and the sum of the
    magnitudes of the terms of each element (for its rounding bound)."""
    x = x.astype(np.float64)
    T, H, D = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(F32(eps)))
        x = x * weight.astype(np.float64)
    y, m = x.copy(), np.abs(x)
    if cos_sin is not None:
        R = cos_sin.shape[1]
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c = cos_sin[positions, i].astype(np.float64)[:, None]
            s = cos_sin[positions, R // 2 + i].astype(np.float64)[:, None]
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
            m[:, :, a] = np.abs(x[:, :, a] * c) + np.abs(x[:, :, b] * s)
            m[:, :, b] = np.abs(x[:, :, b] * c) + np.abs(x[:, :, a] * s)
    return y, m


def decode_pages(cache, cache_dtype, head_dim):
    """A cache as float64 [NB, H, 16, D], without the per-tensor scale."""
    c = cache.cpu()
    if cache_dtype in ("f32", "f16", "bf16"):
        return c.double().numpy()
    if cache_dtype == "e4m3":
        return c.view(torch.float8_e4m3fn).float().double().numpy()
    u = c.numpy()
    NB, H, _ = u.shape
    D = head_dim
    codes = u[:, :, :8 * D].reshape(NB, H, BS, D // 2)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(NB, H, BS, D)
    if cache_dtype == "int4":
        val = np.where(nib >= 8, nib.astype(np.int64) - 16, nib).astype(np.float64)
        sc = np.ascontiguousarray(u[:, :, 8 * D:]).view(np.float32)
        return val * sc.astype(np.float64)[..., None]
    val = np.array([oracle.e2m1_to_double(i) for i in range(16)])[nib]
    sc = np.array([oracle.e4m3_to_double(i) for i in range(256)])
    sc = sc[u[:, :, 8 * D:].reshape(NB, H, BS, D // 16)]
    return val * np.repeat(sc, 16, axis=-1)


def bounds_of(keys):
    """Record of one block and KV head from its written keys [n, D] (float64
    values that fp32 holds): (hi codes, lo codes, scale)."""
    k = keys.astype(F32)
    big = np.finfo(F32).max
    hi = np.fmax.reduce(k, axis=0)
    lo = np.fmin.reduce(k, axis=0)
    none = np.isnan(k).all(0)
    hi = np.clip(np.where(none, 0, hi), -big, big).astype(F32)
    lo = np.clip(np.where(none, 0, lo), -big, big).astype(F32)
    s = F32(max(np.abs(hi).max(), np.abs(lo).max()) / F32(127))
    if s == 0:
        z = np.zeros(len(hi), dtype=np.int8)
        return z, z, F32(0)
    return (np.clip(np.ceil(hi / s), -127, 127).astype(np.int8),
            np.clip(np.floor(lo / s), -127, 127).astype(np.int8), s)


def records(bounds, D):
    """(hi, lo, scale) of a bounds tensor, as numpy."""
    b = bounds.cpu().numpy()
    sc = np.ascontiguousarray(b[..., 2 * D:2 * D + 4]).view(np.float32)[..., 0]
    return b[..., :D].view(np.int8), b[..., D:2 * D].view(np.int8), sc


def tokens_of(md):
    """(token, request, position) of every token of a request."""
    qsl, L = md["query_start_loc"], md["seq_lens"]
    for r in range(len(L)):
        n = qsl[r + 1] - qsl[r]
        for i in range(n):
            yield int(qsl[r] + i), r, int(L[r] - n + i)


def select(q, hi, lo, sc, md, group, K, first, last):
    """q float32 [T, Hq, D] (values of its type); records of the cache.
    Returns {(token, KV head): list of blocks}."""
    T, Hq, D = q.shape
    out = {}
    for t, r, p in tokens_of(md):
        n = p // BS + 1
        for h in range(Hq // group):
            if n <= K:
                out[t, h] = list(range(n))
                continue
            x = q[t, h * group:(h + 1) * group].astype(F32)
            sq = F32(np.abs(x).max() / F32(127))
            if sq > 0:
                code = np.clip(np.rint((x / sq).astype(F32)), -127, 127).astype(np.int64)
            else:
                code = np.zeros(x.shape, dtype=np.int64)
            kept = set(range(first)) | set(range(n - last, n))
            mid = [b for b in range(n) if b not in kept]
            blk = md["block_tables"][r, mid]
            H, L = hi[blk, h].astype(np.int64), lo[blk, h].astype(np.int64)
            dots = (np.maximum(code, 0) @ H.T + np.minimum(code, 0) @ L.T).max(0)
            with np.errstate(over="ignore"):
                score = dots.astype(F32) * sc[blk, h]
            order = sorted(range(len(mid)), key=lambda i: (-score[i], mid[i]))
            out[t, h] = sorted(kept | {mid[i] for i in order[:K - len(kept)]})
    return out


def attend(q, k, v, md, lists, group, scale, k_scale=1.0, v_scale=1.0):
    """q float64 [T, Hq, D]; k, v decoded caches (float64).  Returns (out, sum
    of p |v|, largest sum |q k| scale) per element / row; rows of no list NaN."""
    T, Hq, D = q.shape
    out = np.full((T, Hq, D), np.nan)
    mag = np.zeros((T, Hq, D))
    qk = np.zeros((T, Hq, 1))
    scale, k_scale, v_scale = (float(F32(x)) for x in (scale, k_scale, v_scale))
    req = {t: (r, p) for t, r, p in tokens_of(md)}
    for (t, h), blocks in lists.items():
        r, p = req[t]
        rows = slice(h * group, (h + 1) * group)
        if len(blocks) == 0:
            out[t, rows] = 0
            continue
        b = np.asarray(blocks)
        keep = (b[:, None] * BS + np.arange(BS)).reshape(-1) <= p
        phys = md["block_tables"][r, b]
        kk = k[phys, h].reshape(-1, D)[keep] * k_scale
        vv = v[phys, h].reshape(-1, D)[keep] * v_scale
        x = q[t, rows] @ kk.T * scale
        e = np.exp(x - x.max(-1, keepdims=True))
        pr = e / e.sum(-1, keepdims=True)
        out[t, rows] = pr @ vv
        mag[t, rows] = pr @ np.abs(vv)
        qk[t, rows] = (np.abs(q[t, rows]) @ np.abs(kk).T * abs(scale)).max(-1, keepdims=True)
    return out, mag, qk


def attend_tolerance(ref, mag, qk, out_dtype, prob_dtype):
    """Per element: the output's rounding; each probability's rounding to the
    type that the product takes (half a step of p, so half a step of sum p
    |v|); and the fp32 arithmetic.  The last: a score is a sum of 128 products
    whose partial sums round at 2^-24 of sum |q k| each (a factor 2 for the
    tensor core's alignment), and the products with the scale and log2(e) and
    the exponential add a few 2^-24 of the score: 2^-16 (1 + sum |q k| scale)
    of sum p |v| covers them."""
    return (half(out_dtype) * np.abs(ref) + half(prob_dtype) * mag * (1 + half(out_dtype)) +
            2.0 ** -16 * (1 + qk) * mag + 2.0 ** -24)
