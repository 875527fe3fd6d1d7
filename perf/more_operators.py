"""The operators of decoding with several hypotheses over a paged cache, as they
are measured: cases, inputs, the operators' plain forms in elementary torch
operations, the same calls through this package, and their values in 64 bits.

* beam    -- the best continuations of each group of beams: log-softmax of the
             beams' logits, plus their scores, the K largest over beams and
             vocabulary
* fork    -- rows of a step take over other rows' blocks: block tables, lengths
             and reference counts reordered, blocks without a reference back on
             the stack of free ids, a shared last block replaced by a copy
* copy    -- those copies, for the caches of all layers at once
* compact -- tokens dropped from requests: tables, lengths, references, and the
             list of moves that closes the gaps
* move    -- those moves, for the caches of all layers at once, in place

Where ``own`` is true, ``run`` calls the package; elsewhere the plain forms.
"""
import math

import numpy as np
import torch

own = False

BS = 16
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
       "e4m3": torch.uint8}
_EB = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
_TOP = torch.finfo(torch.float32).max


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request of four beams, a vocabulary of 32000: four short rows
        dict(name="beam 1x4x32000 f32", op="beam", groups=1, width=4, vocab=32000, k=8,
             pad=0, done=0.0, masked=0.0, dtype="f32"),
        # a decode batch of the Llama-3.1-8B vocabulary, finished beams among them
        dict(name="beam 64x4x128256 bf16", op="beam", groups=64, width=4, vocab=128256, k=4,
             pad=0, done=0.1, masked=0.0, dtype="bf16"),
        # wide beams over fp32 logits, twice as many continuations as beams, rows
        # of odd length, a part of the vocabulary masked out
        dict(name="beam 32x8x50257 f32", op="beam", groups=32, width=8, vocab=50257, k=16,
             pad=7, done=0.0, masked=0.3, dtype="f32"),
        # beams of 16 requests between two steps
        dict(name="fork 16x4 512-4096", op="fork", groups=16, width=4, lo=512, hi=4096,
             tail=64, gone=0.0),
        # a large step, some requests ending in it: 1024 rows
        dict(name="fork 128x8 1K-16K", op="fork", groups=128, width=8, lo=1024, hi=16384,
             tail=200, gone=0.1),
        # what 16 requests of four beams copy after a fork, Llama-3.1-8B caches
        dict(name="copy 24 x 32 layers bf16", op="copy", pairs=24, room=64, layers=32,
             blocks=512, hkv=8, d=128, dtype="bf16"),
        # a large step's copies, Llama-3.1-70B caches in FP8
        dict(name="copy 500 x 80 layers e4m3", op="copy", pairs=500, room=512, layers=80,
             blocks=1500, hkv=8, d=128, dtype="e4m3"),
        # the accepted path of a tree of 32 drafted tokens, 64 requests
        dict(name="compact tree 64 x 32", op="compact", reqs=64, lo=512, hi=8192, span=32,
             keep=0.2, shared=0.0),
        # long prompts cut down to the tokens that matter, a few blocks shared
        # with other requests
        dict(name="compact 32 x 2K-32K", op="compact", reqs=32, lo=2048, hi=32768, span=0,
             keep=0.25, shared=0.05),
        # the moves of an accepted path, all layers
        dict(name="move tree 64 x 32 layers bf16", op="move", reqs=64, lo=512, hi=1024,
             span=32, keep=0.2, layers=32, hkv=8, d=128, dtype="bf16"),
        # the moves of cut prompts
        dict(name="move 8 x 4K-8K x 16 layers bf16", op="move", reqs=8, lo=4096, hi=8192,
             span=0, keep=0.5, layers=16, hkv=8, d=128, dtype="bf16"),
        # one long prompt over an FP8 cache with heads of 64 channels
        dict(name="move 1 x 32K x 32 layers e4m3 d64", op="move", reqs=1, lo=32768, hi=32768,
             span=0, keep=0.25, layers=32, hkv=8, d=64, dtype="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["beam", "fork", "copy", "compact", "move"])
    if op == "beam":
        width = rng.choice([1, 2, 3, 4, 5, 8, 16])
        groups = max(1, _log(rng, 1, 256) // width)
        return dict(op=op, groups=groups, width=width, vocab=_log(rng, 1000, 128256),
                    k=rng.choice([width, 2 * width]), pad=rng.choice([0, 0, 1, 63]),
                    done=rng.choice([0.0, 0.2]), masked=rng.choice([0.0, 0.5]),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "fork":
        width = rng.choice([1, 2, 3, 4, 8, 16])
        lo = _log(rng, 1, 2048)
        return dict(op=op, groups=max(1, _log(rng, 1, 512) // width), width=width, lo=lo,
                    hi=_log(rng, lo, 16384), tail=_log(rng, 1, 400),
                    gone=rng.choice([0.0, 0.3]))
    hkv, d = rng.choice([(8, 128), (8, 64), (32, 128), (2, 128), (1, 64), (5, 128)])
    dt = rng.choice(["bf16", "f16", "e4m3", "f32"])
    if op == "copy":
        pairs = _log(rng, 1, 200)
        return dict(op=op, pairs=pairs, room=pairs + rng.randint(0, 100),
                    layers=_log(rng, 1, 40), blocks=2 * pairs + rng.randint(1, 300), hkv=hkv,
                    d=d, dtype=dt)
    lo = _log(rng, 20, 4096)
    span = rng.choice([0, 0, 8, 17, 64])
    if op == "compact":
        reqs = _log(rng, 1, 200)
        return dict(op=op, reqs=reqs, lo=max(lo, span),
                    hi=max(lo, span, min(_log(rng, lo, 32768), 600000 // reqs)), span=span,
                    keep=rng.uniform(0.05, 0.95), shared=rng.choice([0.0, 0.1]))
    reqs, layers = _log(rng, 1, 32), _log(rng, 1, 32)
    most = 150000 * 8 * 128 // (hkv * d * _EB[dt] * reqs * layers)
    return dict(op=op, reqs=reqs, lo=max(min(lo, most), span, 8),
                hi=max(min(_log(rng, lo, 32768), most), min(lo, most), span, 8), span=span,
                keep=rng.uniform(0.05, 0.95), layers=layers, hkv=hkv, d=d, dtype=dt)


def _lens(lo, hi, n):
    """n lengths from lo to hi, spread over their logarithm."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    return np.round(lo * (hi / lo) ** (np.arange(n) / (n - 1))).astype(np.int64)


def _kept(c):
    """(lengths, tokens kept as they are, listed tokens kept) of each request: all
    but the last `span` tokens are kept as they are (span 0: the first four)."""
    lens = _lens(c["lo"], c["hi"], c["reqs"])
    start = np.maximum(lens - c["span"], 0) if c["span"] else np.minimum(lens, 4)
    return lens, start, np.maximum(1, np.round((lens - start) * c["keep"]).astype(np.int64)
                                   ) * (lens > start)


def work(c):
    """Bytes read and written once, and operations, of one pass."""
    op = c["op"]
    if op == "beam":
        rows = c["groups"] * c["width"]
        n = int(round(rows * (1 - c["done"]))) * c["vocab"]
        # logits, beam scores in, scores, parents and tokens out
        return {"bytes": n * _EB[c["dtype"]] + 4 * rows + 12 * c["groups"] * c["k"],
                "flops": 4 * n}
    if op == "fork":
        lens = _lens(c["lo"], c["hi"], c["groups"])
        entries = int(((lens + 15) // BS).sum()) * c["width"]
        rows = c["groups"] * c["width"]
        # tables in and out, a reference count of each distinct block, lengths,
        # sources, the copies' pairs
        return {"bytes": 8 * entries + 8 * entries // c["width"] + 28 * rows, "flops": 0}
    if op == "copy":
        return {"bytes": 4 * c["pairs"] * c["layers"] * c["hkv"] * BS * c["d"] *
                _EB[c["dtype"]] + 16 * c["pairs"], "flops": 0}
    lens, start, k = _kept(c)
    moved = int(k.sum())
    if op == "compact":
        # the list in, two slots out per listed token, the listed part of the
        # tables, reference counts and the freed ids
        blocks = int(((lens + 15) // BS - start // BS).sum())
        return {"bytes": 20 * moved + 12 * blocks + 20 * len(lens), "flops": 0}
    return {"bytes": moved * (4 * c["layers"] * c["hkv"] * c["d"] * _EB[c["dtype"]] + 16),
            "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _pages(gen, layers, blocks, hkv, d, dtype):
    shape = (layers, blocks, hkv, BS, d)
    if dtype == "e4m3":
        # random codes, none of them a NaN
        x = torch.randint(0, 255, shape, generator=gen, device="cuda", dtype=torch.uint8)
        return torch.where((x & 127) == 127, x ^ 1, x)
    return torch.randn(shape, generator=gen, device="cuda", dtype=_DT[dtype])


def _beam_rows(gen, c):
    """Logits of beams that share most of their context, so that a group's rows are
    alike, and the beams' scores."""
    B, W, V = c["groups"], c["width"], c["vocab"]
    dt = _DT[c["dtype"]]
    rand = dict(generator=gen, device="cuda")
    rows = torch.empty(B * W, V + c["pad"], device="cuda", dtype=dt)
    for b in range(B):
        base = torch.randn(V, **rand) * 2.2
        x = base + 0.7 * torch.randn(W, V, **rand)
        if c["masked"]:
            x = torch.where(torch.rand(V, **rand) < c["masked"], -math.inf, x)
        rows[b * W:(b + 1) * W, :V] = x.to(dt)
        rows[b * W:(b + 1) * W, V:] = 99.0
    scores = -(torch.rand(B, W, **rand) * 3 + 2).cumsum(1) * 0.7
    done = torch.rand(B, W, **rand) < c["done"]
    return rows[:, :V], scores, done.to(torch.uint8)


def _fork_tables(rng, c):
    """Tables of groups of beams: a shared prompt, then blocks shared by the beams
    that descend from one another, and each beam's own last blocks."""
    lens = rng.permutation(_lens(c["lo"], c["hi"], c["groups"]))
    B, W = c["groups"], c["width"]
    nb = (lens + BS - 1) // BS
    M = int(nb.max()) + 2
    table = np.full((B * W, M), -1, dtype=np.int64)
    n = 0
    for b in range(B):
        L, k = int(lens[b]), int(nb[b])
        # full blocks of the tokens before the beams parted
        own0 = max(0, (L - int(rng.integers(1, c["tail"] + 1))) // BS)
        row = np.arange(n, n + own0)
        n += own0
        for w in range(W):
            # beams part one after another
            cut = own0 + int(rng.integers(0, (k - own0) // 2 + 1)) if w else own0
            cut = min(cut, L // BS)
            r = b * W + w
            if w:
                table[r, :cut] = table[r - 1, :cut]
            else:
                table[r, :cut] = row
            table[r, cut:k] = np.arange(n, n + k - cut)
            n += k - cut
    pool = int(nb.sum()) * W + 64  # as if nothing were shared
    ids = rng.permutation(pool)
    used = table >= 0
    table[used] = ids[table[used]]
    refs = np.bincount(table[used], minlength=pool)
    src = np.arange(B * W).reshape(B, W)
    for b in range(B):
        p = rng.random(W) ** 2 + 0.05
        src[b] = b * W + np.sort(rng.choice(W, W, p=p / p.sum()))
        if rng.random() < c["gone"]:
            src[b] = -1
    return lens.repeat(W), table, np.maximum(refs - 1, 0), ids[n:], pool, src.reshape(-1)


def _paged_rows(rng, lens, shared):
    """Tables of requests in a random order of blocks; a share of the blocks is
    held by some other request, too."""
    nb = (lens + BS - 1) // BS
    M, n = int(nb.max()), int(nb.sum())
    table = np.full((len(lens), M), -1, dtype=np.int64)
    here = np.arange(M) < nb[:, None]
    free = max(16, int(n * shared * 1.5))
    ids = rng.permutation(n + free)
    table[here] = ids[:n]
    refs = np.zeros(n + free, dtype=np.int64)
    refs[ids[:n]] = rng.random(n) < shared
    return table, refs, ids[n:], n + free


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng([seed, 78])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=c)
    new = lambda *n, t=torch.int32: torch.full(n, -1, device="cuda", dtype=t)  # noqa: E731
    op = c["op"]
    if op == "beam":
        s["logits"], s["scores"], done = _beam_rows(gen, c)
        s["done"] = done if c["done"] else None
        s["end"] = 2 if c["done"] else -1
        B, K = c["groups"], c["k"]
        s["out"] = (torch.empty(B, K, device="cuda"), new(B, K), new(B, K))
        if own:
            import paged_kv_cache_82_gb300 as pa
            s["space"] = torch.empty(pa.pa_beam_select_workspace_size(
                B, c["width"], c["vocab"], K), device="cuda", dtype=torch.uint8)
        return s
    if op == "fork":
        lens, table, refs, free, nb, src = _fork_tables(rng, c)
        R = len(lens)
        stack = np.full(nb, -1)
        stack[:len(free)] = free
        s.update(lens=_i32(lens), table=_i32(table), refs=_i32(refs), stack=_i32(stack),
                 count=_i32([len(free)]), src=_i32(src), table_out=new(*table.shape),
                 lens_out=new(R), refs_out=new(nb), count_out=new(1),
                 pairs=new(R, 2, t=torch.int64), num_pairs=new(1))
        if own:
            import paged_kv_cache_82_gb300 as pa
            s["space"] = torch.empty(pa.pa_fork_blocks_workspace_size(R, table.shape[1]),
                                     device="cuda", dtype=torch.uint8)
        return s
    if op == "copy":
        args = (c["layers"], c["blocks"], c["hkv"], c["d"], c["dtype"])
        s["kc"], s["vc"] = _pages(gen, *args), _pages(gen, *args)
        ids = rng.permutation(c["blocks"])
        pairs = np.full((c["room"], 2), -1, dtype=np.int64)
        pairs[:c["pairs"], 1] = ids[:c["pairs"]]
        # several beams copy one block
        pairs[:c["pairs"], 0] = ids[c["pairs"] + rng.integers(0, c["pairs"], c["pairs"])]
        s["pairs"], s["num_pairs"] = torch.from_numpy(pairs).cuda(), _i32([c["pairs"]])
        return s
    lens, start, k = _kept(c)
    order = rng.permutation(len(lens))
    lens, start, k = lens[order], start[order], k[order]
    K = max(1, int(k.max()))
    keep = np.full((len(lens), K), -1, dtype=np.int64)
    for r in range(len(lens)):
        keep[r, :k[r]] = start[r] + np.sort(rng.choice(lens[r] - start[r], k[r], replace=False))
    table, refs, free, nb = _paged_rows(rng, lens, c.get("shared", 0.0))
    R = len(lens)
    if op == "compact":
        stack = np.full(2 * nb, -1)
        stack[:len(free)] = free
        s.update(lens=_i32(lens), start=_i32(start), k=_i32(k), keep=_i32(keep),
                 table=_i32(table), refs=_i32(refs), stack=_i32(stack),
                 count=_i32([len(free)]), nb=nb, table_out=new(*table.shape),
                 lens_out=new(R), refs_out=new(nb), count_out=new(1),
                 src=new(R, K + BS, t=torch.int64), dst=new(R, K + BS, t=torch.int64),
                 moves=new(R))
        if own:
            import paged_kv_cache_82_gb300 as pa
            s["space"] = torch.empty(pa.pa_compact_blocks_workspace_size(R, table.shape[1]),
                                     device="cuda", dtype=torch.uint8)
        return s
    args = (c["layers"], nb, c["hkv"], c["d"], c["dtype"])
    s["kc"], s["vc"] = _pages(gen, *args), _pages(gen, *args)
    src = np.full((R, K + BS), -1, dtype=np.int64)
    dst = src.copy()
    for r in range(R):
        p, q = keep[r, :k[r]], start[r] + np.arange(k[r])
        src[r, :k[r]] = table[r, p // BS] * BS + p % BS
        dst[r, :k[r]] = table[r, q // BS] * BS + q % BS
    s.update(src=torch.from_numpy(src).cuda(), dst=torch.from_numpy(dst).cuda(), moves=_i32(k))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"beam": _beam, "fork": _fork, "copy": _copy, "compact": _compact,
            "move": _move}[s["case"]["op"]](s)


def _cache_view(x):
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _beam(s):
    c = s["case"]
    B, W, V, K = c["groups"], c["width"], c["vocab"], c["k"]
    if own:
        import paged_kv_cache_82_gb300 as pa
        return list(pa.pa_beam_select(s["logits"], s["scores"], K, finished=s["done"],
                                      end_token=s["end"], scores=s["out"][0],
                                      parents=s["out"][1], tokens=s["out"][2],
                                      workspace=s["space"]))
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=_TOP)
    top = x.amax(1, keepdim=True).clamp(min=-_TOP)
    # sums and scores in 64 bits: two beams' scores can lie next to each other
    mass = (x.double() - top.double()).exp().sum(1, keepdim=True)
    # each beam's K largest logits, equal ones by the lower token: one whole number
    # that orders both
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits)
    key = (key << 32) + (V - torch.arange(V, device="cuda"))
    kk = min(K, V)
    tok = key.topk(kk, 1).indices
    best = x.gather(1, tok)
    cum = s["scores"].reshape(-1, 1)
    best = torch.where(cum.isfinite() & (best > -math.inf),
                       cum.double() + (best.double() - top.double() - mass.log()), -math.inf)
    if s["done"] is not None:
        over = s["done"].reshape(-1, 1) != 0
        first = torch.arange(kk, device="cuda") == 0
        same = torch.where(first & cum.isfinite(), cum.double(), -math.inf)
        best = torch.where(over, same, best)
        tok = torch.where(over, s["end"], tok)
    best = best.view(B, W * kk)
    order = best.sort(dim=1, descending=True, stable=True).indices[:, :K]
    score = best.gather(1, order).float()
    there = score > -math.inf
    parent = order // kk + torch.arange(B, device="cuda")[:, None] * W
    token = tok.view(B, W * kk).gather(1, order)
    gap = K - score.shape[1]
    out = (score, torch.where(there, parent, -1).int(), torch.where(there, token, -1).int())
    pad = torch.nn.functional.pad
    return [pad(out[0], (0, gap), value=-math.inf), pad(out[1], (0, gap), value=-1),
            pad(out[2], (0, gap), value=-1)]


def _push(refs, table, released, stack, base):
    """Blocks whose references ran out (a negative count), in the order in which the
    released entries of the tables name them, onto the stack at `base`; how many."""
    nb, cap = refs.numel(), stack.numel()
    ids = torch.where(released, table, nb).long().flatten()
    flat = torch.arange(ids.numel(), device="cuda")
    first = torch.full((nb + 1,), ids.numel(), device="cuda").scatter_reduce(
        0, ids, flat, "amin")
    spent = torch.nn.functional.pad(refs, (0, 1)) < 0
    owner = spent[ids] & (first[ids] == flat)
    at = torch.where(owner, base + owner.long().cumsum(0) - 1, cap).clamp(max=cap)
    room = torch.nn.functional.pad(stack, (0, 1))
    room.scatter_(0, at, ids.int())
    stack.copy_(room[:cap])
    return owner.sum()


def _fork(s):
    if own:
        import paged_kv_cache_82_gb300 as pa
        pa.pa_fork_blocks(s["src"], s["table"], s["lens"], s["refs"], s["stack"], s["count"],
                          block_tables_out=s["table_out"], seq_lens_out=s["lens_out"],
                          extra_refs_out=s["refs_out"], free_count_out=s["count_out"],
                          block_mapping=s["pairs"], num_pairs=s["num_pairs"],
                          workspace=s["space"])
        return [s["table_out"], s["lens_out"], s["refs_out"], s["stack"], s["count_out"],
                s["pairs"], s["num_pairs"]]
    table, lens, src = s["table"], s["lens"].long(), s["src"].long()
    R, M = table.shape
    nb = s["refs"].numel()
    at = src.clamp(min=0)
    live = src >= 0
    col = torch.arange(M, device="cuda")
    here = col < ((lens + 15) // BS)[:, None]
    uses = torch.zeros(R, device="cuda", dtype=torch.int64).scatter_add(0, at, live.long())
    ids = torch.where(here, table, nb).long()
    refs = torch.nn.functional.pad(s["refs"], (0, 1)).long()
    refs.scatter_add_(0, ids.flatten(), (uses - 1)[:, None].expand(R, M).flatten())
    refs = refs[:nb]
    freed = _push(refs, table, here & (uses == 0)[:, None], s["stack"], s["count"].long())
    top = s["count"].long() + freed
    refs = refs.clamp(min=0)
    # the rows' last blocks, where they are partly filled
    length = torch.where(live, lens[at], 0)
    part = length % BS != 0
    last = torch.where(part, table[at, length // BS], nb).long()
    row = torch.arange(R, device="cuda")
    held = torch.zeros(nb + 1, device="cuda", dtype=torch.int64).scatter_add(
        0, last, torch.ones_like(last))
    first = torch.full((nb + 1,), R, device="cuda").scatter_reduce(0, last, row, "amin")
    others = torch.nn.functional.pad(refs, (0, 1))[last] + 1 - held[last]
    need = part & ~((first[last] == row) & (others <= 0))
    nth = need.long().cumsum(0) - 1
    got = need & (nth < top)
    fresh = s["stack"][(top - 1 - nth).clamp(0, len(s["stack"]) - 1)]
    refs = torch.nn.functional.pad(refs, (0, 1))
    refs.scatter_add_(0, torch.where(got, last, nb), torch.full_like(last, -1))
    moved = table[at]
    moved = torch.where(got[:, None] & (col == (length // BS)[:, None]), fresh[:, None], moved)
    keep = (col < ((length + 15) // BS)[:, None])
    s["table_out"].copy_(torch.where(keep, moved, s["table_out"]))
    pairs = torch.full((R + 1, 2), -1, device="cuda")
    slot = torch.where(got, nth, R)
    pairs.scatter_(0, slot[:, None].expand(R, 2), torch.stack([last, fresh.long()], 1))
    n = got.sum()
    return [s["table_out"], length.int(), refs[:nb].int(), s["stack"],
            (top - n).int().view(1), pairs[:R], n.int().view(1)]


def _copy(s):
    if own:
        import paged_kv_cache_82_gb300 as pa
        pa.pa_copy_blocks_layers(s["kc"], s["vc"], s["pairs"], s["num_pairs"],
                                 cache_dtype=s["case"]["dtype"])
    else:
        # the pairs past the count copy a block onto itself
        on = torch.arange(len(s["pairs"]), device="cuda") < s["num_pairs"]
        src, dst = s["pairs"].unbind(1)
        src, dst = torch.where(on, src, dst[0]), torch.where(on, dst, dst[0])
        src[s["case"]["pairs"]:] = src[0]
        for x in (s["kc"], s["vc"]):
            x.index_copy_(1, dst, x[:, src])
    return [_cache_view(s["kc"]), _cache_view(s["vc"])]


def _compact(s):
    stack = s["stack"].clone()  # (its upper end changes with every pass)
    if own:
        import paged_kv_cache_82_gb300 as pa
        pa.pa_compact_blocks(s["keep"], s["k"], s["table"], s["lens"], s["refs"], stack,
                             s["count"], keep_start=s["start"],
                             block_tables_out=s["table_out"], seq_lens_out=s["lens_out"],
                             extra_refs_out=s["refs_out"], free_count_out=s["count_out"],
                             src_slots=s["src"], dst_slots=s["dst"], num_moves=s["moves"],
                             workspace=s["space"])
        return [s["table_out"], s["lens_out"], s["refs_out"], stack, s["count_out"],
                s["src"], s["dst"], s["moves"]]
    table, lens, start, k = s["table"], s["lens"].long(), s["start"].long(), s["k"].long()
    R, M = table.shape
    nb, K = s["nb"], s["keep"].shape[1]
    n = start + k
    j = torch.arange(K, device="cuda")
    still = (s["keep"] == start[:, None] + j) & (j < k[:, None])
    u = start + still.sum(1)  # tokens that stay where they are
    f = (u // BS)[:, None]
    col = torch.arange(M, device="cuda")
    left, had = ((n + 15) // BS)[:, None], ((lens + 15) // BS)[:, None]
    ids = torch.where(col < had, table, nb).long()
    refs = torch.nn.functional.pad(s["refs"], (0, 1)).long()
    swap = (col >= f) & (col < left) & (refs[ids] > 0)
    need = swap.sum(1)
    runs = need.cumsum(0) <= s["count"]
    swap = swap & runs[:, None]
    nth = swap.flatten().long().cumsum(0).view(R, M) - 1
    fresh = stack[(s["count"].long() - 1 - nth).clamp(0, len(stack) - 1)]
    after = torch.where(swap, fresh, table)
    released = swap | (runs[:, None] & (col >= left) & (col < had))
    refs.scatter_add_(0, torch.where(released, table, nb).long().flatten(),
                      torch.full((R * M,), -1, device="cuda"))
    refs = refs[:nb]
    base = s["count"].long() - swap.sum()
    freed = _push(refs, table, released, stack, base)
    length = torch.where(runs, n, lens)
    keep = col < ((length + 15) // BS)[:, None]
    s["table_out"].copy_(torch.where(keep, after, s["table_out"]))
    # the moves: tokens from the first block that changes on
    i = f * BS + torch.arange(K + BS, device="cuda")
    some = runs[:, None] & (i < n[:, None]) & ((u < n) | swap.any(1))[:, None]
    listed_at = (i - start[:, None]).clamp(0, K - 1)
    pos = torch.where(i < start[:, None], i, s["keep"].long().gather(1, listed_at))
    pos, i = torch.where(some, pos, 0), torch.where(some, i, 0)
    src = table.long().gather(1, pos // BS) * BS + pos % BS
    dst = after.long().gather(1, i // BS) * BS + i % BS
    s["src"].copy_(torch.where(some, src, s["src"]))
    s["dst"].copy_(torch.where(some, dst, s["dst"]))
    return [s["table_out"], length.int(), refs.clamp(min=0).int(), stack,
            (base + freed).int(), s["src"], s["dst"], some.sum(1).int()]


def _move(s):
    if own:
        import paged_kv_cache_82_gb300 as pa
        pa.pa_move_tokens(s["kc"], s["vc"], s["src"], s["dst"], s["moves"],
                          cache_dtype=s["case"]["dtype"])
    else:
        on = torch.arange(s["src"].shape[1], device="cuda") < s["moves"][:, None]
        # the places past a row's moves repeat its first move
        src = torch.where(on, s["src"], s["src"][:, :1]).flatten()
        dst = torch.where(on, s["dst"], s["dst"][:, :1]).flatten()
        for x in (s["kc"], s["vc"]):
            for layer in x:
                layer[dst // BS, :, dst % BS] = layer[src // BS, :, src % BS]
    return [_cache_view(s["kc"]), _cache_view(s["vc"])]


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] != "beam":
        return None  # whole numbers, and values as they were
    s = prepare(case, seed)
    B, W, V, K = c["groups"], c["width"], c["vocab"], c["k"]
    out = torch.full((B, K), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(B):
        logp = torch.log_softmax(s["logits"][b * W:(b + 1) * W].double(), 1)
        logp = logp + s["scores"][b].double()[:, None]
        if s["done"] is not None:
            over = s["done"][b] != 0
            logp[over] = -math.inf
            logp[over, s["end"]] = s["scores"][b][over].double()
        top = logp.flatten().topk(min(K, W * V)).values
        out[b, :len(top)] = top
    return [out, None, None]
