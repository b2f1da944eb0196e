"""spec_beam_select where beams' scores are equal or nearly so: every output is
compared, and what is expected follows from the order that the interface states
(scores, then w * V + v; within a beam the logits)."""

import numpy as np
import pytest
import torch

from rejection_sampling_verifier_amd import binding
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
