"""pa_beam_select on beams that are copies of each other, in rows of any alignment:
equal logits and equal beam scores make equal scores, so the lower beam comes first."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# elements before and behind each row: contiguous ones, then slices of longer ones
LAYOUTS = [(0, 0), (0, 1), (1, 2), (5, 58)]


def _rows(rng, B, V, dtype):
    x = rng.standard_normal((B, V)).astype(np.float32) * np.float32(2.5)
    return torch.from_numpy(x).to(DT[dtype])


def _copies(x, W, lead, trail):
    """Each row of x W times in a row, on the GPU, as slices of longer rows."""
    B, V = x.shape
    whole = torch.full((B * W, lead + V + trail), 50.0, dtype=x.dtype, device="cuda")
    whole[:, lead:lead + V] = x.cuda().repeat_interleave(W, 0)
    return whole[:, lead:lead + V]


def _want(x, W, K):
    """(parents, tokens): larger logits first, then lower beams, then lower tokens."""
    d = x.double().numpy()
    parents, tokens = [], []
    for g, row in enumerate(d):
        best = np.argsort(-row, kind="stable")[:K]
        beam, tok = np.repeat(np.arange(W), len(best)), np.tile(best, W)
        order = np.lexsort((tok, beam, -row[tok]))[:K]
        parents.append(g * W + beam[order])
        tokens.append(tok[order])
    return np.array(parents), np.array(tokens)


def _check(x, W, K, score, layouts):
    parents, tokens = _want(x, W, K)
    cum = torch.full((x.shape[0], W), score, dtype=torch.float32, device="cuda")
    first = None
    for lead, trail in layouts:
        s, p, t = pa.pa_beam_select(_copies(x, W, lead, trail), cum, K)
        where = f"{lead} + V + {trail}"
        np.testing.assert_array_equal(p.cpu().numpy(), parents, err_msg=where)
        np.testing.assert_array_equal(t.cpu().numpy(), tokens, err_msg=where)
        # (all sums were taken again, so that the scores' bits do not depend on where rows
        # lie either)
        first = s if first is None else first
        assert torch.equal(s, first), where
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("V", [37, 701, 9001, 50257, 140003])
def test_copies_in_rows_of_any_alignment(dtype, V):
    rng = np.random.default_rng(V)
    x = _rows(rng, 3, V, dtype)
    # the last pick in the middle of a run of equal scores, and at one's end
    _check(x, 4, 6, -1.5, LAYOUTS)
    _check(x, 4, 8, -0.3, LAYOUTS)
    _check(x, 7, 33, -20.0, LAYOUTS)


@pytest.mark.parametrize("V", [50257, 140003])
@pytest.mark.parametrize("groups", [1, 70, 100, 160])
def test_copies_whatever_the_number_of_groups(groups, V):
    """One, two and four CTAs to a group share the sums that are taken again."""
    rng = np.random.default_rng(groups)
    _check(_rows(rng, groups, V, "f32"), 2, 3, -1.5, [(0, 0), (3, 2)])


def test_copies_among_other_beams():
    """Two pairs of copies a distance apart, not next to each other."""
    rng = np.random.default_rng(5)
    for V in (701, 33001):
        for dtype in sorted(DT):
            x = _rows(rng, 2, V, dtype)
            rows = x[[0, 1, 0, 1]].cuda()
            s, p, t = pa.pa_beam_select(
                rows, torch.tensor([[-1.0, -40.0, -1.0, -40.0]], device="cuda"), 5)
            parents, tokens = _want(x[:1], 2, 5)
            np.testing.assert_array_equal(p.cpu().numpy(), 2 * parents)
            np.testing.assert_array_equal(t.cpu().numpy(), tokens)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_equal_scores_by_logits_and_beam_scores(dtype):
    """Copies whose beam scores lie as far apart as some of their logits do: a lower logit
    of a better beam scores as much as a higher one of a worse beam, and the lower beam
    comes first.  (Logits in steps of 1/4 and beam scores in steps of 1/2, so that their
    sums are exact.)"""
    rng = np.random.default_rng(6)
    for V, W, K, pad in ((37, 4, 30, 1), (701, 5, 64, 0), (20011, 16, 128, 3)):
        x = torch.from_numpy(np.round(rng.standard_normal((4, V)) * 10) / 4).to(DT[dtype])
        cum = rng.choice([-0.5, -1.0, -1.5, -3.0], (4, W)).astype(np.float32)
        s, p, t = pa.pa_beam_select(_copies(x, W, 0, pad), torch.from_numpy(cum).cuda(), K)
        for g, row in enumerate(x.double().numpy()):
            best = np.argsort(-row, kind="stable")[:K]
            beam, tok = np.repeat(np.arange(W), len(best)), np.tile(best, W)
            # (the row's log-sum is the same for all)
            order = np.lexsort((tok, -row[tok], beam, -(cum[g][beam] + row[tok])))[:K]
            np.testing.assert_array_equal(p[g].cpu().numpy(), g * W + beam[order])
            np.testing.assert_array_equal(t[g].cpu().numpy(), tok[order])
    assert pa.pa_get_device_error() == 0
