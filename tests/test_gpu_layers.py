"""pa_copy_blocks_layers and pa_move_tokens, bit by bit, and the calls of a beam step
and of dropped tokens together."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _beam_ref as ref

pytestmark = pytest.mark.gpu

# type: (bytes of a token's channels, bytes of its scales) for head_dim D
ROWS = {"bf16": lambda D: (2 * D, 0), "f16": lambda D: (2 * D, 0), "f32": lambda D: (4 * D, 0),
        "e4m3": lambda D: (D, 0), "int4": lambda D: (D // 2, 4),
        "nvfp4": lambda D: (D // 2, D // 16)}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.uint8}


def _bytes(rng, L, NB, H, D, cache):
    row, scale = ROWS[cache](D)
    return rng.integers(0, 256, (L, NB, H, 16 * (row + scale)), dtype=np.uint8)


def _cache(raw, D, cache):
    """The cache tensor of such bytes, on the GPU."""
    t = torch.from_numpy(raw.copy()).cuda()
    if cache in DT:
        t = t.view(DT[cache]).unflatten(-1, (16, D))
    return t


def _raw(t, shape):
    return t.contiguous().view(torch.uint8).reshape(shape).cpu().numpy()


@pytest.mark.parametrize("cache", sorted(ROWS))
@pytest.mark.parametrize("L,NB,H,D,P", [(1, 7, 1, 64, 3), (3, 40, 8, 128, 11),
                                        (5, 90, 3, 64, 44), (2, 300, 5, 128, 149)])
def test_copied_blocks(cache, L, NB, H, D, P):
    rng = np.random.default_rng(NB)
    k, v = _bytes(rng, L, NB, H, D, cache), _bytes(rng, L, NB, H, D, cache)
    ids = rng.permutation(NB)
    pairs = np.stack([ids[P + rng.integers(0, NB - P, P)], ids[:P]], 1)
    for n in {0, 1, P // 2, P}:
        kc, vc = _cache(k, D, cache), _cache(v, D, cache)
        count = torch.tensor([n], dtype=torch.int32, device="cuda")
        pa.pa_copy_blocks_layers(kc, vc, torch.from_numpy(pairs).cuda(), count,
                                 cache_dtype=cache)
        for got, before in ((kc, k), (vc, v)):
            np.testing.assert_array_equal(_raw(got, before.shape),
                                          ref.copy_blocks(before, pairs[:n]))
    assert pa.pa_get_device_error() == 0


def test_the_same_as_a_call_per_layer_and_single_layers():
    rng = np.random.default_rng(1)
    k, v = _bytes(rng, 3, 20, 4, 128, "bf16"), _bytes(rng, 3, 20, 4, 128, "bf16")
    pairs = torch.tensor([[3, 4], [3, 5], [9, 0]], device="cuda")
    a, b = _cache(k, 128, "bf16"), _cache(v, 128, "bf16")
    c, d, e, f = a.clone(), b.clone(), a.clone(), b.clone()
    pa.pa_copy_blocks_layers(a, b, pairs)
    for layer in range(3):
        pa.pa_copy_blocks(c[layer], d[layer], pairs)
        pa.pa_copy_blocks_layers(e[layer], f[layer], pairs)
    for x in (c, e):
        assert torch.equal(a.view(torch.int16), x.view(torch.int16))
    for x in (d, f):
        assert torch.equal(b.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("cache", ["bf16", "nvfp4"])
def test_layers_of_one_buffer(cache):
    """K and V of a layer next to each other, and layers with a gap between them."""
    rng = np.random.default_rng(2)
    both = _bytes(rng, 8, 12, 2, 128, cache).reshape(4, 2, 12, 2, -1)
    pairs = np.array([[1, 2], [7, 3]])
    src = np.array([[5 * 16 + 3, 5 * 16 + 9]])
    dst = np.array([[5 * 16 + 2, 6 * 16 + 1]])
    want = both.copy()
    row, scale = ROWS[cache](128)
    for i in (0, 1):
        want[:, i] = ref.move_tokens(ref.copy_blocks(both[:, i], pairs), src, dst, [2], row,
                                     scale)
    t = _cache(both, 128, cache)
    moves = torch.tensor([2], dtype=torch.int32, device="cuda")
    dev = [torch.from_numpy(x).cuda() for x in (pairs, src, dst)]
    pa.pa_copy_blocks_layers(t[:, 0], t[:, 1], dev[0], cache_dtype=cache)
    pa.pa_move_tokens(t[:, 0], t[:, 1], dev[1], dev[2], moves, cache_dtype=cache)
    np.testing.assert_array_equal(_raw(t, want.shape), want)
    # every second layer only (from two buffers), the others untouched
    t, u = _cache(both, 128, cache), _cache(both, 128, cache)
    pa.pa_copy_blocks_layers(t[::2, 0], u[::2, 1], dev[0], cache_dtype=cache)
    half = both.copy()
    half[::2, 0] = ref.copy_blocks(both[::2, 0], pairs)
    np.testing.assert_array_equal(_raw(t, half.shape), half)
    half = both.copy()
    half[::2, 1] = ref.copy_blocks(both[::2, 1], pairs)
    np.testing.assert_array_equal(_raw(u, half.shape), half)
    with pytest.raises(pa.PaError):  # K and V the same, or half a layer apart
        pa.pa_copy_blocks_layers(t[:, 0], t[:, 0], dev[0], cache_dtype=cache)
    flat = t.reshape(4, 24, *t.shape[3:])
    with pytest.raises(pa.PaError):
        pa.pa_move_tokens(flat[:, :12], flat[:, 6:18], dev[1], dev[2], moves,
                          cache_dtype=cache)


def test_blocks_and_counts_out_of_range():
    rng = np.random.default_rng(3)
    k = _bytes(rng, 2, 6, 1, 64, "f16")
    pairs = np.array([[0, 6], [-1, 2], [1, 3], [6, 4]])
    for n, flags in ((4, pa.PA_DEV_ERR_BLOCK_ID), (9, pa.PA_DEV_ERR_BLOCK_ID |
                                                   pa.PA_DEV_ERR_METADATA),
                     (-1, pa.PA_DEV_ERR_METADATA)):
        a, b = _cache(k, 64, "f16"), _cache(k, 64, "f16")
        pa.pa_copy_blocks_layers(a, b, torch.from_numpy(pairs).cuda(),
                                 torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert pa.pa_get_device_error() == flags
        want = ref.copy_blocks(k, [(1, 3)] if n > 0 else [])
        np.testing.assert_array_equal(_raw(a, k.shape), want)
        np.testing.assert_array_equal(_raw(b, k.shape), want)


def _gaps(rng, R, per_row, NB):
    """Ascending moves to lower places of each row's own tokens; a row's slots are in
    blocks of its own, in any order."""
    blocks = rng.permutation(NB)[:R * per_row].reshape(R, per_row)
    n = per_row * 16
    src = np.full((R, n + 3), 10 ** 12, np.int64)  # (past the moves: not read)
    dst = src.copy()
    moves = np.zeros(R, np.int32)
    for r in range(R):
        m = int(rng.integers(0, n + 1))
        p, q = np.sort(rng.choice(n, m, replace=False)), np.arange(m)
        src[r, :m] = blocks[r, p // 16] * 16 + p % 16
        dst[r, :m] = blocks[r, q // 16] * 16 + q % 16
        moves[r] = m
    return src, dst, moves


@pytest.mark.parametrize("cache", sorted(ROWS))
@pytest.mark.parametrize("L,H,D,R,per_row", [(1, 1, 64, 1, 1), (2, 1, 128, 3, 9),
                                             (1, 2, 64, 1, 130), (3, 8, 128, 5, 20),
                                             (16, 8, 64, 20, 3), (2, 3, 128, 2, 70)])
def test_moved_tokens(cache, L, H, D, R, per_row):
    """Gaps closed in place: few warps (narrow slices) to many, one step of a warp to
    many."""
    rng = np.random.default_rng(per_row)
    NB = R * per_row + 4
    k, v = _bytes(rng, L, NB, H, D, cache), _bytes(rng, L, NB, H, D, cache)
    src, dst, moves = _gaps(rng, R, per_row, NB)
    kc, vc = _cache(k, D, cache), _cache(v, D, cache)
    pa.pa_move_tokens(kc, vc, *(torch.from_numpy(x).cuda() for x in (src, dst, moves)),
                      cache_dtype=cache)
    assert pa.pa_get_device_error() == 0
    for got, before in ((kc, k), (vc, v)):
        want = ref.move_tokens(before, src, dst, moves, *ROWS[cache](D))
        np.testing.assert_array_equal(_raw(got, before.shape), want)


def test_padding_and_slots_and_counts_out_of_range():
    rng = np.random.default_rng(4)
    k = _bytes(rng, 2, 5, 2, 64, "bf16")
    src = np.array([[3, -1, 9, 80, 12], [20, 21, 22, 23, 24], [40, 40, 40, 40, 40]])
    dst = np.array([[1, 2, -1, 3, 79], [17, 18, 19, 10 ** 15, 20], [41, 42, 43, 44, 45]])
    moves = np.array([5, 4, 6], np.int32)
    a, b = _cache(k, 64, "bf16"), _cache(k, 64, "bf16")
    pa.pa_move_tokens(a, b, *(torch.from_numpy(x).cuda() for x in (src, dst, moves)))
    assert pa.pa_get_device_error() == pa.PA_DEV_ERR_SLOT | pa.PA_DEV_ERR_METADATA
    want = k.copy()
    for s, d in ((3, 1), (12, 79), (20, 17), (21, 18), (22, 19)):
        want[:, d // 16, :, d % 16 * 128:][..., :128] = k[:, s // 16, :, s % 16 * 128:][..., :128]
    np.testing.assert_array_equal(_raw(a, k.shape), want)
    np.testing.assert_array_equal(_raw(b, k.shape), want)


# ---- the calls together ---------------------------------------------------------------
def test_beam_search_in_one_captured_graph():
    """Twenty steps of beam search over a paged cache, replayed from one graph: select,
    fork, copy in all layers, metadata of the new tokens, cache writes.  What each beam's
    table names must be the tokens of its own hypothesis, through every copy."""
    rng = np.random.default_rng(11)
    B, W, V, L, H, D, steps = 3, 4, 500, 3, 2, 64, 40
    R, NB, M = B * W, 200, 12
    prompt = [5, 16, 30]
    # one state per token: the logits of the next one
    trans = torch.randn(V, V, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    trans *= 2
    kc = torch.zeros(L, NB, H, 16, D, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    i32 = dict(dtype=torch.int32, device="cuda")
    # row 0 of each group holds the prompt, the others are idle
    tables, lens = torch.full((R, M), -1, **i32), torch.zeros(R, **i32)
    refs, count = torch.zeros(NB, **i32), torch.zeros(1, **i32)
    ids = rng.permutation(NB).astype(np.int32)
    stack = torch.from_numpy(ids.copy()).cuda()
    used = 0
    history = {}
    for g, n in enumerate(prompt):
        nb = -(-n // 16)
        tables[g * W, :nb] = torch.from_numpy(ids[used:used + nb]).cuda()
        used += nb
        lens[g * W] = n
        hist = [int(x) for x in rng.integers(0, V, n)]
        for j, tok in enumerate(hist):
            b = int(tables[g * W, j // 16])
            kc[:, b, :, j % 16], vc[:, b, :, j % 16] = tok % 256, tok // 256
        history[g * W] = hist
    stack[:NB - used] = torch.from_numpy(ids[used:]).cuda()
    count.fill_(NB - used)
    scores = torch.full((B, W), float("-inf"), device="cuda")
    scores[:, 0] = 0
    done = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    last = torch.zeros(R, dtype=torch.int64, device="cuda")
    for g in range(B):
        last[g * W] = history[g * W][-1]
    END = 3
    ones = torch.ones(R, **i32)
    mapping, pairs = torch.empty(R, 2, dtype=torch.int64, device="cuda"), torch.zeros(1, **i32)
    parents, tokens = torch.empty(B, W, **i32), torch.empty(B, W, **i32)
    log_parents = torch.empty(steps, R, **i32)
    log_tokens = torch.empty(steps, R, **i32)
    log_at = torch.zeros(1, dtype=torch.int64, device="cuda")
    logits = torch.empty(R, V, device="cuda")
    qsl, pos = torch.empty(R + 1, **i32), torch.empty(R, **i32)
    slots = torch.empty(R, dtype=torch.int64, device="cuda")
    work = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        pa.pa_beam_select_workspace_size(B, W, V, W), pa.pa_fork_blocks_workspace_size(R, M))]

    def step():
        torch.index_select(trans, 0, last, out=logits)
        pa.pa_beam_select(logits, scores, W, finished=done, end_token=END, scores=scores,
                          parents=parents, tokens=tokens, finished_out=done, workspace=work[0])
        pa.pa_fork_blocks(parents.view(-1), tables, lens, refs, stack, count,
                          block_mapping=mapping, num_pairs=pairs, workspace=work[1])
        pa.pa_copy_blocks_layers(kc, vc, mapping, pairs)
        pa.pa_build_step(ones, lens, tables, stack, count, NB, R, seq_lens=lens,
                         query_start_loc=qsl, positions=pos, slot_mapping=slots,
                         free_count_out=count)
        tok = tokens.view(-1)
        last.copy_(tok.clamp(min=0))
        rows = tok.view(R, 1, 1).expand(R, H, D)
        k, v = (rows % 256).bfloat16(), (rows // 256).bfloat16()
        for layer in range(L):
            pa.pa_reshape_and_cache(k.contiguous(), v.contiguous(), kc[layer], vc[layer], slots)
        log_parents.index_copy_(0, log_at, parents.view(1, R))
        log_tokens.index_copy_(0, log_at, tokens.view(1, R))
        log_at.add_(1)

    state = [x.clone() for x in (tables, lens, refs, stack, count, scores, done, last, kc, vc,
                                 log_at)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((tables, lens, refs, stack, count, scores, done, last, kc, vc, log_at),
                    state):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    # the same search on the host
    tr = trans.cpu().double().numpy()
    cum = np.full((B, W), -np.inf, np.float32)
    cum[:, 0] = 0
    fin = np.zeros((B, W), np.uint8)
    heads = np.zeros(R, np.int64)
    for g in range(B):
        heads[g * W] = history[g * W][-1]
    hist = {r: history.get(r, []) for r in range(R)}
    for t in range(steps):
        s, p, tok = ref.beam_select(tr[heads], cum, W, fin, END)
        np.testing.assert_array_equal(log_parents[t].cpu().numpy(), p.reshape(-1), str(t))
        np.testing.assert_array_equal(log_tokens[t].cpu().numpy(), tok.reshape(-1))
        hist = {r: hist[p.reshape(-1)[r]] + [int(tok.reshape(-1)[r])] for r in range(R)}
        cum = s.astype(np.float32)
        fin = (tok == END).astype(np.uint8)
        heads = tok.reshape(-1).astype(np.int64)
    assert lens.tolist() == [len(hist[r]) for r in range(R)]
    table, free = tables.cpu().numpy(), stack.cpu().numpy()[:int(count)]
    holders = np.zeros(NB, int)
    for r in range(R):
        for b in table[r, :-(-len(hist[r]) // 16)]:
            holders[b] += 1
    # every block is free or held, and counted so
    assert len(set(free)) == len(free) and (holders[free] == 0).all()
    assert (holders > 0).sum() + len(free) == NB
    np.testing.assert_array_equal(refs.cpu().numpy(), np.maximum(holders - 1, 0))
    kh, vh = kc.float().cpu().numpy(), vc.float().cpu().numpy()
    for r in range(R):
        for j, tok in enumerate(hist[r]):
            b = table[r, j // 16]
            got = kh[:, b, :, j % 16] + 256 * vh[:, b, :, j % 16]
            assert (got == tok).all(), (r, j)
    # all requests end: everything is free again
    pa.pa_fork_blocks(torch.full((R,), -1, **i32), tables, lens, refs, stack, count)
    assert int(count) == NB and not lens.any() and not refs.any()
    assert sorted(stack.tolist()) == list(range(NB)) and pa.pa_get_device_error() == 0


def test_dropped_tokens_then_attention():
    """Tokens dropped in place: attention over what is left equals attention over those
    tokens written to a cache of their own."""
    rng = np.random.default_rng(12)
    B, Hq, H, D, NB = 5, 8, 2, 128, 400
    lens = np.array([700, 33, 16, 1200, 64])
    nb = -(-lens // 16)
    ids = rng.permutation(NB)
    table = np.zeros((B, int(nb.max())), np.int32)
    at = 0
    for r in range(B):
        table[r, :nb[r]] = ids[at:at + nb[r]]
        at += nb[r]
    gen = torch.Generator("cuda").manual_seed(5)
    kc, vc = (torch.randn(2, NB, H, 16, D, device="cuda", generator=gen).bfloat16()
              for _ in range(2))
    q = torch.randn(B, Hq, D, device="cuda", generator=gen).bfloat16()
    refs = np.zeros(NB, np.int32)
    refs[table[0, :9]] = 1                 # a prefix that another request holds, too
    old_k, old_v = kc.clone(), vc.clone()
    keep = np.full((B, 900), -1, np.int32)
    ks = np.zeros(B, np.int32)
    for r in range(B):
        ks[r] = max(1, lens[r] * 2 // 3)
        keep[r, :ks[r]] = np.sort(rng.choice(lens[r], ks[r], replace=False))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    tables, sl, stack, count = i32(table), i32(lens), i32(np.r_[ids[at:], [0] * at]), i32([NB - at])
    src, dst, moves = pa.pa_compact_blocks(i32(keep), i32(ks), tables, sl, i32(refs), stack,
                                           count)
    pa.pa_move_tokens(kc, vc, src, dst, moves)
    qsl = i32(np.arange(B + 1))
    for layer in range(2):
        got = pa.pa_attention(q, kc[layer], vc[layer], tables, sl, qsl, 1, 1200, 0.1)
        # the kept tokens, in pages of their own
        k2, v2 = torch.zeros_like(kc[layer]), torch.zeros_like(vc[layer])
        t2 = np.zeros((B, 60), np.int32)
        n = 0
        for r in range(B):
            m = -(-int(ks[r]) // 16)
            t2[r, :m] = np.arange(n, n + m)
            n += m
            pos, j = keep[r, :ks[r]], np.arange(ks[r])
            b, d = table[r, pos // 16], t2[r, j // 16]
            for new, old in ((k2, old_k[layer]), (v2, old_v[layer])):
                new[d, :, j % 16] = old[b, :, pos % 16]
        want = pa.pa_attention(q, k2, v2, i32(t2), i32(ks), qsl, 1, 900, 0.1)
        assert torch.equal(got, want)
    # what the other request reads is as it was
    assert torch.equal(kc[:, table[0, :9]], old_k[:, table[0, :9]])
    assert sl.tolist() == ks.tolist() and pa.pa_get_device_error() == 0
