"""spec_beam_select and spec_beam_reorder on the GPU against the float64 oracle:
vocabularies that end inside a chunk, ties, near ties between beams, finished,
missing and invalid beams, strides, both types."""

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import beam as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev, f64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def check(logits, scores, finished=None, end=-1, label="", **kw):
    """Tokens and ancestors are exact wherever two beams' candidates are further
    apart than float64 sums can be off (1e-12).  Scores: the logarithm of a sum
    that is off by 2^-20 relative, and half a step of float32."""
    got = binding.beam_select(logits, scores, finished, end=end, **kw)
    torch.cuda.synchronize()
    host = None if finished is None else finished.cpu().numpy()
    tokens, anc, out, fin, margin = ref.beam_select(f64(logits), f64(scores), host, end)
    W = scores.shape[1]
    sure = margin > 1e-12
    say(f"[beam] {label}: {int(sure.sum())} of {len(sure)} sequences, smallest margin {margin.min():.2e}")
    np.testing.assert_array_equal(got[0].cpu().numpy()[sure], tokens[sure])
    np.testing.assert_array_equal(got[1].cpu().numpy().reshape(-1, W)[sure], anc.reshape(-1, W)[sure])
    np.testing.assert_array_equal(got[3].cpu().numpy()[sure], fin[sure])
    s = f64(got[2])
    alive = np.isfinite(out)
    assert (np.isfinite(s) == alive).all() and (s[~alive] == -np.inf).all()
    out = np.where(alive, out, 0.0)
    assert (np.abs(s - out)[alive] <= 2.0 ** -20 + 2.0 ** -24 * np.abs(out[alive])).all()
    return got


def make(B, W, V, dtype, seed=0, first=False, spread=3.0):
    rng = np.random.default_rng(seed)
    logits = dev(rng.standard_normal((B, W, V)) * spread, dtype)
    scores = -np.sort(rng.random((B, W)) * 3 + 10, -1).astype(np.float32)
    if first:
        scores[:, 1:] = -np.inf
    return logits, dev(scores)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [1, 3, 8, 63, 500, 2047, 2048, 2049, 8191, 8200, 40001])
@pytest.mark.parametrize("B,W", [(1, 1), (2, 4), (3, 17)])
def test_vocabularies(dtype, V, B, W):
    check(*make(B, W, V, dtype, V), label=f"B={B} W={W} V={V} {dtype}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("W", [1, 2, 8, 33, 64])
def test_beams(dtype, W):
    check(*make(2, W, 9001, dtype, W), label=f"W={W} {dtype}")


def test_large_batch():
    check(*make(70, 16, 5003, BF16), label="70 sequences")


@pytest.mark.parametrize("V", [50, 20000])
def test_first_step(V):
    """One beam is there: its W best ids."""
    check(*make(3, 8, V, FP32, first=True), label="first step")


@pytest.mark.parametrize("W,V", [(4, 3000), (64, 9000), (8, 8)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_equal_logits(dtype, W, V):
    """Every candidate of a beam has the same score: the lowest ids, and with equal
    scores the lowest beams."""
    logits = torch.full((2, W, V), 1.25, dtype=dtype, device="cuda")
    scores = torch.full((2, W), -4.0, device="cuda")
    tokens, anc, _, _ = binding.beam_select(logits, scores)
    flat = np.arange(W)
    want_v, want_w = flat % V, flat // V
    np.testing.assert_array_equal(tokens.cpu().numpy(), np.tile(want_v, (2, 1)))
    np.testing.assert_array_equal(anc.cpu().numpy().reshape(2, W), np.stack([want_w, W + want_w]))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_equal_rows_at_different_alignments(dtype):
    """Equal beams tie exactly, wherever their rows lie: ids in the order of the beams."""
    rng = np.random.default_rng(9)
    V, W = 5001, 4
    row = dev(rng.standard_normal(V) * 3, dtype)
    buf = torch.empty(W * (V + 1) + 8, dtype=dtype, device="cuda")
    logits = torch.as_strided(buf, (1, W, V), (W * (V + 1), V + 1, 1), 3)
    logits[:] = row
    scores = torch.full((1, W), -2.5, device="cuda")
    tokens, anc, _, _ = binding.beam_select(logits, scores)
    best = int(np.argsort(-f64(row), kind="stable")[0])
    assert tokens.cpu().tolist() == [[best] * W] and anc.cpu().tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("seed", range(6))
def test_near_ties_between_beams(seed):
    """Rows whose best ids lie within 1e-7 of each other after the logarithm of the
    sum (below what float32 sums could tell): the order of the float64 sums."""
    rng = np.random.default_rng(seed)
    B, W, V = 8, 4, 30011
    x = rng.standard_normal((B, W, V)).astype(np.float32) * 2
    scores = np.zeros((B, W), np.float32)
    for b in range(B):
        for w in range(W):
            lp = ref.log_softmax(x[b, w].astype(np.float64))
            # the best id's score moved to -9 - 2e-8 k, as near as float32 allows
            x[b, w, 0] = 0.0
            at = int(np.argmax(lp))
            lp = ref.log_softmax(x[b, w].astype(np.float64))
            scores[b, w] = np.float32(-9.0 - lp[at])
    check(dev(x), dev(scores), label=f"near ties {seed}")


def test_finished_beams():
    rng = np.random.default_rng(4)
    logits, scores = make(6, 5, 700, FP32)
    done = dev((rng.random((6, 5)) < 0.5).astype(np.int32) * 7)
    got = check(logits, scores, done, end=3, label="finished")
    assert got[3].sum() > 0
    done.fill_(1)  # all of them: they stay, best first
    got = check(logits, scores, done, end=699, label="all finished")
    assert (got[0] == 699).all() and (got[2] == scores).all()


def test_end_token_finishes():
    logits, scores = make(2, 3, 100, FP32)
    logits[:, :, 17] = 30.0
    got = check(logits, scores, end=17, label="end")
    assert (got[0][:, 0] == 17).all() and (got[3][:, 0] == 1).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_invalid_beams_give_nothing(bad):
    logits, scores = make(3, 4, 9000, FP32)
    logits[0, 1, 8999] = bad
    logits[1, :, 5] = bad
    scores[2, 0] = bad
    got = check(logits, scores, label=f"{bad}")
    assert (got[0][1] == -1).all() and (got[1].view(3, 4)[1] == -1).all()
    assert (got[2][1] == -float("inf")).all() and (got[3][1] == 0).all()


def test_masked_ids_are_never_chosen():
    """A grammar leaves three ids: fewer candidates than beams at the first step."""
    logits, scores = make(2, 6, 4000, BF16, first=True)
    keep = torch.zeros(4000, dtype=torch.bool, device="cuda")
    keep[[5, 77, 3999]] = True
    logits.masked_fill_(~keep, -float("inf"))
    got = check(logits, scores, label="masked")
    assert (got[0][:, 3:] == -1).all()
    logits.fill_(-float("inf"))
    assert (binding.beam_select(logits, scores)[0] == -1).all()


def test_rows_of_missing_beams_are_not_read():
    logits, scores = make(2, 4, 3000, FP32, first=True)
    logits[:, 1:] = float("nan")
    check(logits, scores, label="NaN in missing beams")


def test_extreme_logits():
    """The largest and smallest numbers, denormals, one dominant id."""
    logits, scores = make(1, 3, 2500, FP32)
    logits[0, 0] = -3e38
    logits[0, 0, 7] = 3e38
    logits[0, 1] *= 1e-42
    logits[0, 2, 100] = 500.0
    check(logits, scores, label="extremes")


@pytest.mark.parametrize("shape,dtype", [((8, 4), torch.float32), ((8, 3), torch.float32), ((8, 5), torch.uint8),
                                         ((8, 3), BF16), ((8, 70001), torch.int32), ((8, 2, 4096), torch.float16),
                                         ((8, 0), torch.int32), ((1, 9), torch.int64)])
def test_reorder(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    state = torch.randint(0, 100, shape, generator=g, device="cuda").to(dtype)
    anc = torch.tensor([3, 3, 0, -1, 7, 6, 100, 2][:shape[0]] if shape[0] > 1 else [0], dtype=torch.int32, device="cuda")
    out = binding.beam_reorder(state, anc)
    ok = (anc >= 0) & (anc < shape[0])
    want = torch.where(ok.view(-1, *[1] * (len(shape) - 1)), state[anc.clamp(0, shape[0] - 1).long()], 0)
    assert torch.equal(out, want.to(dtype))


def test_reorder_of_strided_rows():
    buf = torch.arange(6 * 40, dtype=torch.int32, device="cuda").view(6, 40)
    out = torch.full((6, 64), -1, dtype=torch.int32, device="cuda")
    anc = torch.tensor([5, 4, 3, 2, 1, 0], dtype=torch.int32, device="cuda")
    binding.beam_reorder(buf[:, 3:30], anc, out=out[:, 1:28])
    assert torch.equal(out[:, 1:28], buf.flip(0)[:, 3:30]) and (out[:, 28:] == -1).all() and (out[:, 0] == -1).all()
