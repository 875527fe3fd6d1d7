"""The largest sizes of the calls for several hypotheses, and calls on other streams."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _beam_ref as ref
from tests.test_gpu_beam import DT, _check, _logits, _scores
from tests.test_gpu_fork import _compact, _fork, _i32, _lists, _tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,W,V,K", [
    ("f16", 1, 1, 1 << 24, 128), ("bf16", 1, 3, (1 << 24) - 1, 5), ("f32", 1, 64, 200001, 128),
    ("bf16", 2, 64, 128256, 128), ("f32", 3, 5, 128256, 128), ("f16", 1000, 1, 700, 2),
    ("bf16", 4000, 2, 33, 8)])
def test_largest_selections(dtype, B, W, V, K):
    rng = np.random.default_rng(V % 1000 + K)
    _check(_logits(rng, B * W, V, dtype), _scores(rng, B, W), K)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_equal_logits_of_many_beams(dtype):
    """Every score of a group is equal but for the beam's: more candidates at the last
    pick's score than any list holds."""
    x = torch.zeros(64, 70001).to(DT[dtype])
    scores = np.zeros((1, 64), np.float32)
    _check(x, scores, 128)
    scores[0, 40] = 1.0
    _check(x, scores, 100)


@pytest.mark.parametrize("K", [7, 64, 128])
def test_more_equal_scores_than_a_list_holds(K):
    """One group whose candidates come in many pieces: equal rows, rows of two or three
    values, few allowed tokens, finished beams, beams with nothing to offer, and beams whose
    scores are a power of two apart, as their logits are."""
    rng = np.random.default_rng(K)
    V = 100_001
    x = torch.zeros(6, V)
    x[1] = torch.from_numpy(rng.integers(0, 2, V).astype(np.float32))
    x[2] = torch.from_numpy(rng.integers(0, 3, V).astype(np.float32)) * 0.25
    x[3, 5:] = torch.finfo(torch.float32).min
    x[4] = float("-inf")
    scores = np.array([[-1.0, -1.0, -1.5, -2.0, 0.0, -1.0]], np.float32)
    finished = np.array([[0, 0, 0, 0, 0, 1]], np.uint8)
    _check(x, scores, K, finished, 9)
    _check(x, scores, K)
    _check(x[:4].repeat(16, 1), -np.arange(64, dtype=np.float32)[None] / 8, K)
    one = torch.full((4, V), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16)
    for r in range(4):
        one[r, int(rng.integers(0, V))] = 3.0      # one allowed token of each beam
    _check(one, np.array([[0.0, -1.0, -1.0, -7.5]], np.float32), K)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("allowed", [300, 1500, 6000, 14000])
def test_few_warps_hold_everything(dtype, allowed):
    """Allowed tokens next to each other, the others at the type's lowest value or -inf;
    logits that fall or rise along the vocabulary."""
    rng = np.random.default_rng(allowed)
    V = 50_003
    for rest in (-np.inf, torch.finfo(DT[dtype]).min):
        x = _logits(rng, 8, V, dtype)
        for r in range(8):
            at = int(rng.integers(0, V - allowed))
            x[r, :at], x[r, at + allowed:] = rest, rest
        for K in (3, 40, 128):
            _check(x, _scores(rng, 2, 4), K)
    x = _logits(rng, 8, V, dtype)
    for up in (True, False):
        y = torch.sort(x.float(), 1, descending=not up)[0].to(DT[dtype])
        y[:, allowed::allowed] = torch.finfo(DT[dtype]).min
        for K in (5, 100):
            _check(y, _scores(rng, 2, 4), K)
    trend = torch.log1p(torch.arange(V) / 50.0) * -2
    _check((x.float() + trend).to(DT[dtype]), _scores(rng, 4, 2), 16)


def test_infinite_among_the_largest():
    """More largest numbers than a list holds, and +inf, which counts as one of them."""
    x = torch.zeros(2, 30_000)
    x[0, 2000:7000] = torch.finfo(torch.float32).max
    x[0, 6000:6010] = float("inf")
    x[1, ::3] = float("inf")
    x[1, 1::3] = torch.finfo(torch.float32).max
    x[1, 2::9] = float("nan")
    for K in (1, 8, 100):
        _check(x, np.array([[0.0, -1.0]], np.float32), K)


@pytest.mark.parametrize("in_place", [True, False])
def test_one_row_of_a_million_blocks(in_place):
    rng = np.random.default_rng(1)
    c = _tree(rng, 1, 2, 0, 0)
    n = 1 << 20
    c["table"] = np.full((2, n + 3), -7, np.int32)
    ids = rng.permutation(n + 9).astype(np.int32)
    c["table"][0, :n] = ids[:n]
    c["table"][1, :2] = ids[:2]
    c["lens"] = np.array([16 * n - 5, 32], np.int32)
    c["refs"] = np.zeros(n + 9, np.int32)
    c["refs"][ids[:2]] = 1
    c["stack"] = np.full(n + 9, -5, np.int32)
    c["stack"][:9] = ids[n:]
    c["count"] = 9
    assert not _fork(c, [0, 0], in_place)["flags"]
    assert not _fork(c, [1, -1], in_place)["flags"]      # a million blocks onto the stack
    keep = np.sort(rng.choice(16 * n - 5, 200_000, replace=False)).astype(np.int32)[None]
    keep = np.repeat(keep, 2, 0)
    want = _compact(c, keep, np.array([200_000, -1], np.int32), in_place=in_place)
    assert not want["flags"]


def test_caches_and_layers_beyond_32_bits():
    """Two layers of 5 GB each in K, and in V: places past 2^32 bytes in a layer, and a
    second layer past 2^32."""
    L, NB, H, D = 2, 160_000, 8, 128
    k = torch.empty(L, NB, H, 16, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k[0].numel() * 2 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    near = [0, 1, 2, 131_071, 131_072, 131_073, NB - 2, NB - 1]
    for t in (k, v):
        t[:, near] = torch.randn(L, len(near), H, 16, D, device="cuda", generator=g).bfloat16()
    k0, v0 = k[:, near].clone(), v[:, near].clone()
    pairs = torch.tensor([[NB - 1, 1], [0, NB - 2], [131_072, 131_071]], device="cuda")
    pa.pa_copy_blocks_layers(k, v, pairs)
    src = torch.tensor([[16 * (NB - 1) + 15, 16 * 131_073 + 7],
                        [16 * 131_072 + 4, 2 * 16 + 1]], device="cuda")
    dst = torch.tensor([[16 * 131_073 + 1, 16 * 131_073 + 2],
                        [5, 16 * (NB - 1) + 3]], device="cuda")
    pa.pa_move_tokens(k, v, src, dst, torch.tensor([2, 2], dtype=torch.int32, device="cuda"))
    assert pa.pa_get_device_error() == 0
    for t, t0 in ((k, k0), (v, v0)):
        want = t0.clone()
        want[:, 1], want[:, 6], want[:, 3] = t0[:, 7], t0[:, 0], t0[:, 4]
        want[:, 5, :, 1], want[:, 5, :, 2] = t0[:, 7, :, 15], t0[:, 5, :, 7]
        want[:, 0, :, 5], want[:, 7, :, 3] = t0[:, 4, :, 4], t0[:, 2, :, 1]
        assert torch.equal(t[:, near], want)


def test_calls_at_the_same_time():
    """Each call of a beam step and of dropped tokens on a stream of its own, many times,
    in buffers of its own: the results of the calls alone."""
    rng = np.random.default_rng(9)
    c = _tree(rng, 60, 4, 900, 9, spare=4000)
    src = np.sort(rng.integers(0, 4, (60, 4)), 1) + np.arange(60)[:, None] * 4
    d = _tree(rng, 50, 2, 700, 4000, spare=4000)
    keep, ks, start = _lists(rng, d, 0.4)
    x = _logits(rng, 32, 50000, "bf16").cuda()
    scores = torch.from_numpy(_scores(rng, 8, 4)).cuda()
    fork = [_i32(c[k]) for k in ("table", "lens", "refs", "stack")] + [_i32([c["count"]])]
    comp = [_i32(d[k]) for k in ("table", "lens", "refs", "stack")] + [_i32([d["count"]])]
    sources, kd, kl, st = _i32(src.reshape(-1)), _i32(keep), _i32(ks), _i32(start)
    slots = torch.full((2, len(ks), keep.shape[1] + 16), -1, dtype=torch.int64, device="cuda")
    NB = len(d["refs"])
    cache = torch.randn(3, NB, 2, 16, 64, device="cuda").bfloat16()

    def calls():
        return [[t.clone() for t in fork], [t.clone() for t in comp], slots.clone(),
                cache.clone(), cache.clone() + 1]

    def select(s):
        return pa.pa_beam_select(x, scores, 9)

    def forked(s):
        return (*pa.pa_fork_blocks(sources, *s[0]), *s[0])

    def dropped(s):
        out = pa.pa_compact_blocks(kd, kl, *s[1], keep_start=st, src_slots=s[2][0],
                                   dst_slots=s[2][1])
        pa.pa_move_tokens(s[3], s[4], *out)
        return (*out, *s[1], s[3], s[4])

    works = (select, forked, dropped, select, dropped, forked)
    alone = []
    for w in works:
        alone.append(w(calls()))
        torch.cuda.synchronize()
    states = [[calls() for _ in range(4)] for _ in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    got = [[] for _ in works]
    for i in range(4):
        for j, w in enumerate(works):
            with torch.cuda.stream(streams[j]):
                got[j].append(w(states[j][i]))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for one, many in zip(alone, got):
        for some in many:
            for a, b in zip(one, some):
                assert torch.equal(a, b)


def test_rows_far_apart():
    """A row stride past 2^31 elements in all."""
    rng = np.random.default_rng(12)
    x = _logits(rng, 4, 3001, "bf16")
    rows = torch.empty(4, 1 << 30, dtype=torch.bfloat16, device="cuda")[:, 5:3006]
    rows.copy_(x)
    _check(x, _scores(rng, 2, 2), 5, rows=rows)


@pytest.mark.parametrize("which", range(1, 16))
def test_some_of_the_state_in_place(which):
    """Each of tables, lengths, references and count in place or not, from unaligned
    starts."""
    rng = np.random.default_rng(which)
    names = ("block_tables", "seq_lens", "extra_refs", "free_count")

    def offset(x, value=None):  # the same, four bytes behind a 16-byte boundary
        t = torch.empty(x.numel() + 1, dtype=torch.int32, device="cuda")[1:].view(x.shape)
        return t.copy_(x) if value is None else t.fill_(value)

    for call in ("fork", "compact"):
        c = _tree(rng, 20, 3, 300, 500, spare=900)
        state = [offset(_i32(c[k])) for k in ("table", "lens", "refs", "stack")]
        state.append(_i32([c["count"]]))
        ins = dict(zip(names, (state[0], state[1], state[2], state[4])))
        outs = {n + "_out": offset(ins[n], -9) for i, n in enumerate(names) if which >> i & 1}
        before = np.full_like(c["table"], -9) if which & 1 else c["table"]
        if call == "fork":
            src = rng.integers(-1, 60, 60)
            mapping, pairs = pa.pa_fork_blocks(_i32(src), *state, **outs)
            want = ref.fork(src, c["table"], c["lens"], c["refs"], c["stack"], c["count"], before)
            assert int(pairs) == want["num_pairs"]
            np.testing.assert_array_equal(mapping.cpu().numpy(), want["pairs"])
        else:
            keep, ks, start = _lists(rng, c, 0.3)
            got = pa.pa_compact_blocks(_i32(keep), _i32(ks), *state, keep_start=_i32(start),
                                       **outs)
            want = ref.compact(keep, ks, start, c["table"], c["lens"], c["refs"], c["stack"],
                               c["count"], got[0].cpu().numpy(), got[1].cpu().numpy(), before)
            np.testing.assert_array_equal(got[0].cpu().numpy(), want["src"])
            np.testing.assert_array_equal(got[1].cpu().numpy(), want["dst"])
            np.testing.assert_array_equal(got[2].cpu().numpy(), want["moves"])
        assert pa.pa_get_device_error() == 0 and not want["flags"]
        for n, k in zip(names[:3], ("table", "seq_lens", "refs")):
            np.testing.assert_array_equal(outs.get(n + "_out", ins[n]).cpu().numpy(), want[k])
        np.testing.assert_array_equal(state[3].cpu().numpy(), want["stack"])
        assert int(outs.get("free_count_out", ins["free_count"])) == want["count"]


@pytest.mark.parametrize("R", [120, 150, 190, 230, 270, 330, 500, 800, 1300, 1900, 2600, 4096])
def test_wide_tables_of_few_blocks(R):
    """Rows' state and tiles of tables in shared memory, from little of it to all."""
    rng = np.random.default_rng(R)
    c = _tree(rng, R // 2, 2, 70, 9, spare=R * 5)
    wide = np.full((R, 40_000 if R < 600 else 3000), -7, np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    src = np.sort(rng.integers(0, 2, (R // 2, 2)), 1) + np.arange(R // 2)[:, None] * 2
    assert not _fork(c, src.reshape(-1))["flags"]
    keep, ks, start = _lists(rng, c, 0.3)
    assert _compact(c, keep, ks, start)["flags"] <= {"blocks"}


def test_rows_cut_to_their_first_tokens():
    """No lists at all: keep of no columns."""
    rng = np.random.default_rng(2)
    c = _tree(rng, 9, 2, 200, 300, spare=300)
    start = np.array([int(rng.integers(0, n + 1)) for n in c["lens"]], np.int32)
    for in_place in (True, False):
        assert not _compact(c, np.zeros((18, 0), np.int32), np.zeros(18, np.int32), start,
                            in_place)["flags"]


def test_one_token_to_many_slots():
    k = torch.randn(2, 6, 3, 16, 64, device="cuda").bfloat16()
    v = torch.randn_like(k)
    src = torch.tensor([[5, 5, 5, 90, 5, 7]], device="cuda")
    dst = torch.tensor([[5, 17, 90, 91, 95, 3]], device="cuda")
    k0, v0 = k.clone(), v.clone()
    # (90 is a destination before it is a source: not a list of moves, left out)
    src[0, 3] = -1
    pa.pa_move_tokens(k, v, src, dst, torch.tensor([6], dtype=torch.int32, device="cuda"))
    assert pa.pa_get_device_error() == 0
    for t, t0 in ((k, k0), (v, v0)):
        want = t0.clone()
        for s, d in ((5, 17), (5, 90), (5, 95), (7, 3)):
            want[:, d // 16, :, d % 16] = t0[:, s // 16, :, s % 16]
        assert torch.equal(t, want)
