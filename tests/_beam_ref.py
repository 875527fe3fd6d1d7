"""Plain references of beam selection, forked and compacted rows, block copies and
token moves: loops over the definitions of pa.h, in 64 bits."""
import numpy as np

TOP = float(np.finfo(np.float32).max)


def beam_select(logits, beam_scores, K, finished=None, end_token=-1):
    """logits float64 [B * W, V] (the values of the tensor's type).  (scores float64
    [B, K], parents, tokens)."""
    B, W = beam_scores.shape
    scores = np.full((B, K), -np.inf)
    parents = np.full((B, K), -1, np.int32)
    tokens = np.full((B, K), -1, np.int32)
    for g in range(B):
        cands = []  # (score, beam, logit, token)
        for w in range(W):
            cum = float(beam_scores[g, w])
            if not np.isfinite(cum):
                continue
            if finished is not None and finished[g, w]:
                cands.append((cum, w, 0.0, end_token))
                continue
            x = np.where(np.isnan(logits[g * W + w]), -np.inf, logits[g * W + w])
            x = np.minimum(x, TOP)
            m = x.max()
            if m == -np.inf:
                continue
            s = cum + ((x - m) - np.log(np.exp(x - m).sum()))
            best = np.lexsort((np.arange(len(x)), -x))[:K]
            cands += [(s[t], w, x[t], t) for t in best if x[t] > -np.inf]
        with np.errstate(over="ignore"):
            cands = [c for c in cands if np.float32(c[0]) > -np.inf]
        cands.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        for k, (s, w, _, t) in enumerate(cands[:K]):
            scores[g, k], parents[g, k], tokens[g, k] = s, g * W + w, t
    return scores, parents, tokens


def _free(refs, released, stack, count, flags):
    """Pushes the blocks of the released entries whose count fell below 0."""
    pushed = {}  # (in order)
    for b in released:
        if refs[b] < 0 and b not in pushed:
            if refs[b] < -1:
                flags.add("metadata")
            pushed[b] = True
    for b in pushed:
        refs[b] = 0
        if count < len(stack):
            stack[count] = b
            count += 1
        else:
            flags.add("metadata")
    return count


def _state(table, lens, refs, stack, count):
    R, M = table.shape
    flags = set()
    L = []
    for n in lens:
        ok = 0 <= n <= 16 * M
        if not ok:
            flags.add("metadata")
        L.append(int(n) if ok else 0)
    if not 0 <= count <= len(stack):
        flags.add("metadata")
        count = 0
    return R, L, refs.astype(np.int64), stack.copy(), int(count), flags


def fork(sources, table, lens, refs, stack, count, table_out=None):
    """A dict of what pa_fork_blocks leaves; table_out: the output's contents before
    (the table itself where None)."""
    R, L, refs, stack, count, flags = _state(table, lens, refs, stack, count)
    NB = len(refs)
    blocks = [-(-n // 16) for n in L]
    src = []
    for r, s in enumerate(sources):
        if not -1 <= s < R:
            flags.add("metadata")
            s = r
        src.append(int(s))
    released = []
    for s in range(R):
        uses = src.count(s)
        if uses == 1:
            continue
        for b in table[s, :blocks[s]]:
            if not 0 <= b < NB:
                flags.add("block id")
                continue
            refs[b] += uses - 1
            if uses == 0:
                released.append(int(b))
    count = _free(refs, released, stack, count, flags)
    out = (table if table_out is None else table_out).copy()
    part = []
    for r, s in enumerate(src):
        b = -1
        if s >= 0 and L[s] % 16:
            b = int(table[s, L[s] // 16])
            if not 0 <= b < NB:
                flags.add("block id")
                b = -1
        part.append(b)
    need = []
    for r, b in enumerate(part):
        if b < 0:
            continue
        others = max(refs[b], 0) + 1 - part.count(b)
        if others > 0 or b in part[:r]:
            need.append(r)
    pairs, last = [], {}
    for r in need:
        if not count:
            flags.add("blocks")
            break
        count -= 1
        fresh = int(stack[count])
        if not 0 <= fresh < NB:
            flags.add("block id")
        pairs.append((part[r], fresh))
        refs[part[r]] -= 1
        last[r] = fresh
    new_lens = np.zeros(R, np.int32)
    for r, s in enumerate(src):
        n = L[s] if s >= 0 else 0
        new_lens[r] = n
        row = table[s, :-(-n // 16)].copy()
        if r in last:
            row[-1] = last[r]
        out[r, :len(row)] = row
    mapping = np.full((R, 2), -1, np.int64)
    if pairs:
        mapping[:len(pairs)] = pairs
    return dict(table=out, seq_lens=new_lens, refs=refs.astype(np.int32), stack=stack,
                count=count, pairs=mapping, num_pairs=len(pairs), flags=flags)


def compact(keep, keep_lens, start, table, lens, refs, stack, count, src, dst,
            table_out=None):
    """A dict of what pa_compact_blocks leaves; src, dst: the lists before."""
    R, L, refs, stack, count, flags = _state(table, lens, refs, stack, count)
    NB = len(refs)
    old = refs.copy()
    src, dst = src.copy(), dst.copy()
    out = (table if table_out is None else table_out).copy()
    moves, new_lens = np.zeros(R, np.int32), np.array(L, np.int32)
    released, pops, serving = [], 0, True
    for r in range(R):
        k, s = int(keep_lens[r]), 0 if start is None else int(start[r])
        row = table[r]
        had = -(-L[r] // 16)
        ok = 0 <= lens[r] <= 16 * table.shape[1] and k <= keep.shape[1]
        ok = ok and (k < 0 or 0 <= s <= L[r])
        if ok and k > 0:
            v = [int(x) for x in keep[r, :k]]
            ok = all(a < b for a, b in zip([s - 1] + v, v + [L[r]]))
        if not ok:
            flags.add("metadata")
        new = row[:had].copy()
        if ok and k >= 0:
            n = s + k
            kept = list(range(s)) + [int(x) for x in keep[r, :k]]
            u = 0
            while u < n and kept[u] == u:
                u += 1
            first, left = u // 16, -(-n // 16)
            bad = [b for b in row[first:left] if not 0 <= b < NB]
            swap = [c for c in range(first, left)
                    if 0 <= row[c] < NB and old[row[c]] > 0]
            if bad:
                flags.add("block id")
            serving = serving and pops + len(swap) <= count
            if not serving:
                if pops + len(swap) > count:
                    flags.add("blocks")
            else:
                new = row[:left].copy()
                for c in swap:
                    new[c] = stack[count - 1 - pops]
                    pops += 1
                    if not 0 <= new[c] < NB:
                        flags.add("block id")
                        new[c] = -1
                gone = [c for c in range(first, had) if c in swap or c >= left]
                released += [int(row[c]) for c in gone if 0 <= row[c] < NB]
                new_lens[r] = n
                if u < n or first in swap:
                    moves[r] = n - 16 * first
                    for i, j in enumerate(range(16 * first, n)):
                        a, b = int(row[kept[j] // 16]), int(new[j // 16])
                        fine = 0 <= a < NB and 0 <= b < NB
                        src[r, i] = a * 16 + kept[j] % 16 if fine else -1
                        dst[r, i] = b * 16 + j % 16 if fine else -1
                        if not fine:
                            flags.add("block id")
        out[r, :len(new)] = new
    for b in released:
        refs[b] -= 1
    count = _free(refs, released, stack, count - pops, flags)
    return dict(table=out, seq_lens=new_lens, refs=refs.astype(np.int32), stack=stack,
                count=count, src=src, dst=dst, moves=moves, flags=flags)


# ---- caches as arrays of bytes [L, NB, H, page bytes] -----------------------------
def copy_blocks(cache, pairs):
    """pairs distinct: all sources as they were."""
    out = cache.copy()
    for s, d in pairs:
        out[:, d] = cache[:, s]
    return out


def move_tokens(cache, src, dst, moves, row_bytes, scale_bytes=0):
    """One move after another."""
    out = cache.copy()
    for r in range(len(moves)):
        for a, b in zip(src[r, :moves[r]], dst[r, :moves[r]]):
            if a < 0 or b < 0:
                continue
            for base, w in ((0, row_bytes), (16 * row_bytes, scale_bytes)):
                i, j = base + a % 16 * w, base + b % 16 * w
                out[:, b // 16, :, j:j + w] = out[:, a // 16, :, i:i + w]
    return out
