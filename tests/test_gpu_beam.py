"""pa_beam_select against a plain loop in 64 bits: which tokens, exactly; scores to
the rounding of fp32 and what the kernel's sums may be off.

A score's error: half a step of fp32 (2^-24 of it) and the log of a sum of fp32
exponentials: 2^-22 (the exponential) + ln 2 x 2^-23 x log2 V (the roundings of its
argument, whose mean size is below log2 V) + 18 x 2^-24 (the additions) + 2^-22
(chunks joined)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _beam_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _sum_error(V):
    return 2.0 ** -22 + math.log(2) * 2.0 ** -23 * math.log2(max(V, 2)) \
        + 18 * 2.0 ** -24 + 2.0 ** -22


def _check(x, scores, K, finished=None, end=-1, rows=None, **kw):
    """x: logits on the CPU, rows: on the GPU (x's where None); the call and the
    reference compared."""
    B, W = scores.shape
    rows = x.cuda() if rows is None else rows
    fin = None if finished is None else torch.from_numpy(finished).cuda()
    out_fin = torch.full((B, K), 7, dtype=torch.uint8, device="cuda")
    got = pa.pa_beam_select(rows, torch.from_numpy(scores).cuda(), K, finished=fin,
                            end_token=end, finished_out=out_fin, **kw)
    want = ref.beam_select(x.double().numpy(), scores, K, finished, end)
    s, p, t = (g.cpu().numpy() for g in got)
    np.testing.assert_array_equal(p, want[1])
    np.testing.assert_array_equal(t, want[2])
    there = want[1] >= 0
    assert (s[~there] == -np.inf).all()
    err = np.abs(s[there] - want[0][there])
    bound = 2.0 ** -24 * np.abs(want[0][there]) + _sum_error(x.shape[1])
    assert (err <= bound).all(), float((err - bound).max())
    np.testing.assert_array_equal(out_fin.cpu().numpy(), (t >= 0) & (t == end))
    assert pa.pa_get_device_error() == 0
    return s, p, t


def _logits(rng, rows, V, dtype, scale=2.5):
    return torch.from_numpy(rng.standard_normal((rows, V)).astype(np.float32) * scale).to(
        DT[dtype])


def _scores(rng, B, W):
    return -np.sort(rng.uniform(0, 8, (B, W)).astype(np.float32), axis=1)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B,W,V,K", [
    (1, 1, 1, 1), (1, 1, 5, 3), (1, 1, 3, 8), (2, 3, 7, 5), (1, 4, 257, 8), (3, 2, 2047, 4),
    (2, 4, 2048, 9), (1, 5, 2049, 16), (1, 1, 40000, 128), (1, 64, 1003, 128), (5, 8, 8191, 16),
    (24, 4, 32000, 8), (40, 4, 8193, 7), (8, 16, 50257, 33), (1, 2, 300001, 64)])
def test_shapes(dtype, B, W, V, K):
    rng = np.random.default_rng(B * 1000 + V + K)
    _check(_logits(rng, B * W, V, dtype), _scores(rng, B, W), K)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("pad,first", [(1, 0), (7, 3), (8, 1), (0, 5), (29, 2)])
def test_rows_of_any_stride_and_alignment(dtype, pad, first):
    """Rows that are slices of longer ones, whose other elements must not be read."""
    rng = np.random.default_rng(pad)
    for V, rows in ((1001, 6), (9001, 80)):
        whole = _logits(rng, rows, V + pad + first, dtype)
        whole[:, :first] = 1000.0
        whole[:, first + V:] = float("nan")
        here = slice(first, first + V)
        _check(whole[:, here], _scores(rng, rows // 2, 2), 6, rows=whole.cuda()[:, here])


def test_equal_logits_go_to_the_lower_token():
    """Runs of equal logits longer than the kernel's list, of one value and of few."""
    for V in (3000, 20000):
        x = torch.zeros(4, V)
        _check(x, np.array([[-1.0, -2.0], [-3.0, -3.5]], np.float32), 20)
        x[:, 5::7] = 1.0
        _check(x, np.array([[-1.0, -2.0], [-3.0, -3.5]], np.float32), 100)
        x[:, ::2] = -0.0
        _check(x.bfloat16(), np.array([[-1.0, -2.0], [-3.0, -3.5]], np.float32), 128)
    rng = np.random.default_rng(1)
    coarse = torch.from_numpy(rng.integers(0, 3, (160, 9000)).astype(np.float32))
    _check(coarse, _scores(rng, 40, 4), 12)


def test_beams_that_are_copies_of_each_other():
    """Equal scores to the last bit: the lower beam, for each token."""
    rng = np.random.default_rng(2)
    for V in (700, 33000):
        x = _logits(rng, 1, V, "f32").repeat(4, 1)
        s, p, _ = _check(x, np.full((1, 4), -1.5, np.float32), 8)
        assert p[0].tolist() == [0, 1, 2, 3] * 2
    # more candidates tie than the list of the joining kernel holds
    x = torch.zeros(64, 17000)
    _check(x, np.full((1, 64), -1.0, np.float32), 128)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_scores_closer_than_fp32_sums_resolve(dtype):
    """Two beams whose best scores differ by 1e-8 to 1e-6, either way, by beam scores
    set so: the order is the 64-bit one's."""
    rng = np.random.default_rng(3)
    V = 30011
    for trial in range(6):
        x = _logits(rng, 2, V, dtype, scale=1.0 + trial)
        d = x.double().numpy()
        m = d.max(1)
        logp = -np.log(np.exp(d - m[:, None]).sum(1))
        # beam 0's score is 0: its best log-probability decides; beam 1's is as close
        # as fp32 numbers of this size get
        want = logp[0] - logp[1]
        cum = np.array([[0.0, want]], np.float32)
        for step in range(-2, 3):
            c = cum.copy()
            for _ in range(abs(step)):
                c[0, 1] = np.nextafter(c[0, 1], np.float32(np.sign(step) * 1e9))
            _check(x, c, 1)
            _check(x, c, 5)


@pytest.mark.parametrize("V", [40001, 140003])
def test_close_scores_of_long_rows(V):
    """The same where several CTAs share the sums that are taken again; of several
    groups, some need it."""
    rng = np.random.default_rng(V)
    x = _logits(rng, 12, V, "f32")
    d = x.double().numpy()
    m = d.max(1)
    logp = -np.log(np.exp(d - m[:, None]).sum(1))
    cum = np.zeros((4, 3), np.float32)
    for g in range(4):
        cum[g] = (logp[3 * g] - logp[3 * g:3 * g + 3]).astype(np.float32)
    cum[1] = [-1.0, -2.5, -7.0]
    for step in (-1, 0, 1):
        c = cum.copy()
        c[::2, 1] = np.nextafter(c[::2, 1], np.float32(step * 1e9)) if step else c[::2, 1]
        _check(x, c, 1)
        _check(x, c, 6)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_sorted_logits_and_the_largest_lists(dtype):
    """A vocabulary in the order of its logits (one warp has all the largest), and as
    many continuations as there may be."""
    rng = np.random.default_rng(12)
    x = torch.sort(_logits(rng, 8, 50000, dtype).float(), 1, descending=True)[0].to(DT[dtype])
    _check(x, _scores(rng, 2, 4), 8)
    _check(x.flip(1).contiguous(), _scores(rng, 2, 4), 128)
    x = _logits(rng, 96, 9000, dtype)
    _check(x, _scores(rng, 24, 4), 128)
    _check(x, _scores(rng, 3, 32) * 0.01, 128)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_few_tokens_left_by_masks(dtype):
    """Constrained decoding: a few tokens allowed, the others at -inf or at the type's
    lowest value; fewer and more of them than continuations."""
    rng = np.random.default_rng(13)
    for V, rows in ((9000, 8), (20000, 60)):
        for left in (1, 3, 300):
            for mask in (float("-inf"), torch.finfo(DT[dtype]).min):
                x = _logits(rng, rows, V, dtype)
                allowed = torch.zeros(V, dtype=torch.bool)
                allowed[torch.from_numpy(rng.choice(V, left, replace=False))] = True
                x[:, ~allowed] = mask
                if mask != float("-inf") and left < 8:
                    # (masked tokens' scores differ by less than a 64-bit number of their
                    # size resolves: one beam, so that only tokens decide)
                    _check(x, _scores(rng, rows, 1), 8)
                else:
                    _check(x, _scores(rng, rows // 4, 4), 8)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_masked_infinite_and_nan_logits(dtype):
    rng = np.random.default_rng(4)
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(DT[dtype]).min
    for V in (50, 5000, 20000):
        x = _logits(rng, 12, V, dtype)
        x[0] = -inf                       # nothing left
        x[1] = nan
        x[2, 3:] = -inf                   # fewer than K left
        x[3] = low                        # the type's lowest value everywhere
        x[4, 1:] = low
        x[5, 7] = nan
        x[6, 9] = inf                     # one token forced
        x[7, [1, 4]] = inf
        x[8, ::2] = -inf
        x[9, 11:] = nan
        x[10, :] = inf
        for K in (1, 4, 12):
            _check(x, _scores(rng, 3, 4), K)
            _check(x, _scores(rng, 12, 1), K)


def test_huge_logits():
    rng = np.random.default_rng(5)
    for scale in (1e3, 1e5, 3e8, 1e20, 1e30, 1e38):
        x = torch.from_numpy(rng.standard_normal((4, 3000)).astype(np.float32))
        x = (x * scale).clamp(-3e38, 3e38)
        x[1] -= x[1].max()
        s = np.zeros((2, 2), np.float32)
        got = pa.pa_beam_select(x.cuda(), torch.from_numpy(s).cuda(), 1)
        want = ref.beam_select(x.double().numpy(), s, 1)
        np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
        np.testing.assert_array_equal(got[2].cpu().numpy(), want[2])
        np.testing.assert_allclose(got[0].cpu().numpy(), want[0], rtol=2.0 ** -23,
                                   atol=_sum_error(3000))


def test_beams_that_offer_nothing_and_finished_ones():
    rng = np.random.default_rng(6)
    inf = np.inf
    for V in (900, 12000):
        x = _logits(rng, 32, V, "bf16")
        s = _scores(rng, 8, 4)
        s[0, 1:] = -inf                   # a first step: one beam is alive
        s[1] = -inf                       # none
        s[2, 0] = np.nan
        s[3, 2] = inf
        _check(x, s, 8)
        done = np.zeros((8, 4), np.uint8)
        done[0, 0] = done[2, 1] = done[4] = 1
        done[5, 1:3] = 9
        s[5, 1] = s[5, 2]                 # two finished beams of one score
        s[6, 0] = -inf
        done[6, 0] = 1                    # finished, and nothing offered
        x[16:20] = float("nan")           # a finished beam's logits are not looked at
        for end in (0, 2, V - 1):
            _check(x, s, 4, done, end)
            _check(x, s, 7, done != 0, end)


def test_outputs_in_place_and_given():
    rng = np.random.default_rng(7)
    x, s = _logits(rng, 12, 5000, "f16"), _scores(rng, 3, 4)
    done = np.zeros((3, 4), np.uint8)
    done[1, 2] = 1
    want = ref.beam_select(x.double().numpy(), s, 4, done, 3)
    sd, fd = torch.from_numpy(s).cuda(), torch.from_numpy(done).cuda()
    work = torch.empty(pa.pa_beam_select_workspace_size(3, 4, 5000, 4), dtype=torch.uint8,
                       device="cuda")
    p = torch.empty(3, 4, dtype=torch.int32, device="cuda")
    got = pa.pa_beam_select(x.cuda(), sd, 4, finished=fd, end_token=3, scores=sd, parents=p,
                            finished_out=fd, workspace=work)
    assert got[0] is sd and got[1] is p
    np.testing.assert_array_equal(p.cpu().numpy(), want[1])
    np.testing.assert_array_equal(got[2].cpu().numpy(), want[2])
    np.testing.assert_allclose(sd.cpu().numpy(), want[0], rtol=2.0 ** -23, atol=4e-6)
    np.testing.assert_array_equal(fd.cpu().numpy(), want[2] == 3)


def test_same_bits_from_run_to_run_and_in_any_batch():
    rng = np.random.default_rng(8)
    x, s = _logits(rng, 64, 40000, "bf16").cuda(), torch.from_numpy(_scores(rng, 16, 4)).cuda()
    a = pa.pa_beam_select(x, s, 8)
    for _ in range(3):
        for u, v in zip(a, pa.pa_beam_select(x, s, 8)):
            assert torch.equal(u, v)
    # (other chunk sizes: the same picks)
    one = pa.pa_beam_select(x[20:24], s[5:6], 8)
    assert torch.equal(one[1] + 20, a[1][5:6]) and torch.equal(one[2], a[2][5:6])


def test_other_streams_and_graphs():
    """A call on a stream of its own, and two captured ones with separate workspaces."""
    rng = np.random.default_rng(9)
    xs = [_logits(rng, 8, 9000, "f32") for _ in range(2)]
    s = _scores(rng, 2, 4)
    side = torch.cuda.Stream()
    dev = [x.cuda() for x in xs]
    sd = torch.from_numpy(s).cuda()
    torch.cuda.synchronize()
    got = pa.pa_beam_select(dev[0], sd, 4, stream=side)
    side.synchronize()
    want = [ref.beam_select(x.double().numpy(), s, 4) for x in xs]
    np.testing.assert_array_equal(got[2].cpu().numpy(), want[0][2])
    graphs, outs = [], []
    for x in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pa.pa_beam_select(x, sd, 4))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        np.testing.assert_array_equal(o[1].cpu().numpy(), w[1])
        np.testing.assert_array_equal(o[2].cpu().numpy(), w[2])
