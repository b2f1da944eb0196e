"""spec_beam_select where beams' scores are equal or nearly so: every output is
compared, and what is expected follows from the order that the interface states
(scores, then w * V + v; within a beam the logits)."""

import numpy as np
import pytest
import torch

from oracle import beam as ref
from rejection_sampling_verifier_amd import binding
from test_oracle_beam_ties import in_whole_numbers
from tree_helpers import dev

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def rows(got, b, W):
    """(token, beam, score, finished) of sequence b's outputs."""
    tokens, anc, scores, fin = (t.cpu() for t in got)
    return list(zip(tokens[b].tolist(), (anc.view(-1, W)[b] - b * W).tolist(), scores[b].tolist(), fin[b].tolist()))


# ---- no row is left to be summed: all beams finished, missing or invalid

@pytest.mark.parametrize("W", [2, 8, 33, 64])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_finished_beams_with_equal_scores(W, dtype):
    """They stay, in the order of the beams; every output is written by one round of the selection."""
    B, V = 200, 700
    g = torch.Generator(device="cuda").manual_seed(W)
    logits = torch.randn((B, W, V), generator=g, device="cuda").to(dtype)
    scores = torch.full((B, W), -3.25, device="cuda")
    scores[1::2, W // 2:] = -1.5  # the later half is better there
    done = torch.ones((B, W), dtype=torch.int32, device="cuda")
    for _ in range(5):
        got = binding.beam_select(logits, scores, done, end=4)
        for b in (0, 1, B - 2, B - 1):
            order = list(range(W)) if b % 2 == 0 else list(range(W // 2, W)) + list(range(W // 2))
            assert rows(got, b, W) == [(4, w, float(scores[b, w]), 1) for w in order]
        assert torch.equal(got[0][2::2], got[0][:1].expand(B // 2 - 1, W))
        assert torch.equal(got[2][2::2], got[2][:1].expand(B // 2 - 1, W))
        assert torch.equal(got[2][3::2], got[2][1:2].expand(B // 2 - 1, W))


@pytest.mark.parametrize("bad", [float("nan"), INF, None])
def test_finished_beams_beside_beams_without_candidates(bad):
    """Two finished beams within a float32 step of each other; the others are missing, or their logits invalid."""
    B, W, V = 64, 6, 3000
    logits = torch.zeros((B, W, V), device="cuda")
    scores = torch.full((B, W), -2.0, device="cuda")
    if bad is None:
        scores[:] = -INF
    else:
        logits[:, :, 11] = bad
    scores[:, 1], scores[:, 4] = -2.0, float(np.nextafter(np.float32(-2.0), np.float32(0.0)))
    done = torch.zeros((B, W), dtype=torch.int32, device="cuda")
    done[:, 1] = done[:, 4] = 1
    for _ in range(5):
        got = binding.beam_select(logits, scores, done, end=7)
        want = [(7, 4, float(scores[0, 4]), 1), (7, 1, -2.0, 1)]
        for b in (0, 31, B - 1):
            assert rows(got, b, W)[:2] == want
        assert (got[0][:, 2:] == -1).all() and (got[1].view(B, W)[:, 2:] == -1).all()
        assert (got[2][:, 2:] == -INF).all() and (got[3][:, 2:] == 0).all()


# ---- equal scores of different beams

def order_of(got, b, W):
    return [r[:2] for r in rows(got, b, W)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_the_lower_beam_comes_first(dtype):
    logits = torch.full((1, 2, 9), -1.0, dtype=dtype, device="cuda")
    logits[..., 0] = 0.0
    got = binding.beam_select(logits, torch.tensor([[-1.0, -2.0]], device="cuda"))
    assert order_of(got, 0, 2) == [(0, 0), (1, 0)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("W,V,levels", [(4, 50, 10), (8, 3000, 40), (16, 20000, 60), (8, 20000, 2)])
def test_shared_rows_of_whole_numbers(dtype, W, V, levels):
    """Beams of one row each with scores that are whole numbers apart: many candidates are equal, from a few
    to more than a workgroup ranks at once."""
    rng = np.random.default_rng(V + levels)
    B = 12
    x = np.stack([np.maximum(-rng.permutation(V), -levels) for _ in range(B)])
    scores = rng.integers(-6, 0, (B, W))
    logits = dev(np.repeat(x[:, None], W, 1).astype(np.float32), dtype)
    got = binding.beam_select(logits, dev(scores.astype(np.float32)))
    host = ref.beam_select(logits.double().cpu().numpy(), scores.astype(np.float64))
    for b in range(B):
        want = in_whole_numbers(x[b], scores[b], W)
        assert order_of(got, b, W) == want, b
        assert list(zip(host[0][b].tolist(), (host[1].reshape(-1, W)[b] - b * W).tolist())) == want, b


@pytest.mark.parametrize("finished_first", [True, False])
def test_finished_beside_live(finished_first):
    """A live beam with one id left has it at its own score."""
    logits = torch.full((1, 2, 5), -INF, device="cuda")
    logits[..., 3] = 4.0
    scores = torch.full((1, 2), -2.0, device="cuda")
    done = torch.tensor([[1, 0]] if finished_first else [[0, 1]], dtype=torch.int32, device="cuda")
    got = binding.beam_select(logits, scores, done, end=1)
    want = [(1, 0, -2.0, 1), (3, 1, -2.0, 0)] if finished_first else [(3, 0, -2.0, 0), (1, 1, -2.0, 1)]
    assert rows(got, 0, 2) == want


def test_logits_decide_within_a_beam():
    """1e-30 and 0 are equal beside a largest logit of 5, as scores; -0 and 0 are equal logits."""
    logits = torch.full((1, 4, 20), -INF, device="cuda")
    logits[0, 0, [2, 5, 10, 11]] = torch.tensor([5.0, -0.0, 1e-30, 0.0], device="cuda")
    got = binding.beam_select(logits, torch.tensor([[-1.0, -INF, -INF, -INF]], device="cuda"))
    assert order_of(got, 0, 4) == [(2, 0), (10, 0), (5, 0), (11, 0)]


# ---- the scores themselves

@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [2, 8, 2049, 40001])
@pytest.mark.parametrize("gap", [1, 6, 17, 25, 30])
def test_scores_of_confident_rows(dtype, V, gap):
    """One id has nearly all of the probability: what the others have is kept.  The bound: each of their
    exponentials is off by 2^-20 relative at most, which moves the logarithm by that much of their share;
    float64 sums and logarithms (2^-50); half a step of float32."""
    rng = np.random.default_rng(gap)
    B = 3
    x = rng.standard_normal((B, 1, V)) * 0.25 - gap
    x[np.arange(B), 0, rng.integers(0, V, B)] = 0.125
    logits = dev(x, dtype)
    got = binding.beam_select(logits, torch.zeros((B, 1), device="cuda"))
    y = logits.double().cpu().numpy()[:, 0]
    top = y.max(-1)
    rest = np.exp(y - top[:, None])
    rest[np.arange(B), y.argmax(-1)] = 0.0
    rest = rest.sum(-1)
    want = -np.log1p(rest)
    err = np.abs(got[2].double().cpu().numpy()[:, 0] - want)
    assert (err <= 2.0 ** -20 * rest / (1 + rest) + 2.0 ** -50 + 2.0 ** -24 * np.abs(want)).all(), (err, want)


# ---- nearer than float32 exponentials tell

@pytest.mark.parametrize("seed", range(3))
def test_scores_apart_by_less_than_the_exponentials_error(seed):
    """Two beams whose rows differ by a few float32 steps everywhere, with the same largest logit and score: their best candidates are apart
    by their logarithms' difference alone, set to 4e-11 by a logit of little mass.  Half of the time the second
    beam is the better one."""
    rng = np.random.default_rng(seed)
    B, V = 48, 30011
    x = (rng.standard_normal((B, 1, V)) * 2 * (1 + 1e-6 * rng.standard_normal((B, 2, V)))).astype(np.float32)
    x[:, :, 0] = 3.0
    x[:, :, 5] = 12.0  # far above the others, so that the best candidates of both are this id
    want = 4e-11 * np.where(rng.random(B) < 0.5, 1, -1)
    for b in range(B):
        for _ in range(3):  # Newton's steps on row 1's first logit
            lse = [np.log(np.exp(x[b, w].astype(np.float64) - 12.0).sum()) for w in range(2)]
            p = np.exp(float(x[b, 1, 0]) - 12.0 - lse[1])
            x[b, 1, 0] = np.float32(x[b, 1, 0] + np.log1p((lse[0] - want[b] - lse[1]) / p))
    scores = np.full((B, 2), -3.0, np.float32)
    tokens, anc, out, _, margin = ref.beam_select(x.astype(np.float64), scores.astype(np.float64))
    assert (tokens == 5).all() and (margin > 1e-11).all() and (margin < 1e-10).all(), margin
    assert 8 < (anc.reshape(B, 2)[:, 0] % 2).sum() < 40
    got = binding.beam_select(dev(x), dev(scores))
    np.testing.assert_array_equal(got[0].cpu().numpy(), tokens)
    np.testing.assert_array_equal(got[1].cpu().numpy(), anc)
    assert (np.abs(got[2].double().cpu().numpy() - out) <= 2.0 ** -24 * np.abs(out) + 2.0 ** -45).all()
