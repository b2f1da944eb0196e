"""spec_latent_prompt on rows of very different sizes: values far beyond and far
below float16's range, in rows that a token sees and in rows that it does not
(later ones, other requests')."""

import numpy as np
import pytest
import torch

import test_gpu_latent_prompt as pro
from rejection_sampling_verifier_amd import binding
from tree_helpers import f64

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def same(a, b):
    """Equal bit for bit, NaN included."""
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def make(lens, new, H=2, dims=(64, 32, 64, 128), **kw):
    """Keys are made of the first half of the latent part, values of the second, so
    that rows' values can be of any size beside ordinary scores."""
    s = pro.make(lens, new, H=H, dims=dims, **kw)
    half = dims[3] // 2
    s["w_k"][:, :, half:] = 0
    s["w_v"][:, :, :half] = 0
    s["half"], s["R"] = half, dims[3]
    return s


def values_of(s, b, j):
    """The part of row j of sequence b that its values are made of."""
    ps = s["cache"].shape[1]
    return s["cache"][s["table"][b, j // ps].long(), j % ps, s["half"]:s["R"]]


def resize(s, b, rng, lo, hi):
    """Every row of sequence b times a power of two."""
    for j in range(int(s["lens"][b])):
        values_of(s, b, j).mul_(2.0 ** int(rng.integers(lo, hi + 1)))


# (lens, new), heads, dims: few and many query tiles; both tiles of the expansion; heads whose values lie in one to
# three of the parts that their sizes are found in
SHAPES = [((150, 61), (150, 20), 2, (64, 32, 64, 128)), ((300, 41), (300, 41), 3, (128, 64, 128, 512)),
          ((200, 90), (70, 90), 5, (80, 32, 72, 256)), ((400, 100), (400, 100), 70, (64, 32, 64, 128)),
          ((700, 3, 1497), (9, 3, 5), 130, (64, 32, 72, 136)), ((140,), (140,), 7, (96, 64, 96, 384)),
          ((130, 70), (130, 70), 30, (8, 8, 8, 16)), ((200, 90), (200, 90), 80, (128, 64, 128, 512)),
          ((200, 90), (200, 90), 80, (80, 32, 120, 256)), ((700, 1503), (5, 9), 130, (64, 32, 104, 136))]


@pytest.mark.parametrize("dtype,lo,hi", [(BF16, -40, 40), (BF16, -100, -60), (FP16, -10, 10)])
@pytest.mark.parametrize("lens,new,H,dims", SHAPES)
def test_rows_of_all_sizes(lens, new, H, dims, dtype, lo, hi):
    s = make(lens, new, H=H, dims=dims, dtype=dtype)
    rng = np.random.default_rng(H)
    for b in range(len(lens)):
        resize(s, b, rng, lo, hi)
    pro.check(s, f"{lens} {H} heads {dims} {dtype} 2^{lo} to 2^{hi}")


@pytest.mark.parametrize("dtype,by", [(BF16, 2.0 ** 36), (BF16, 1e30), (FP16, 3e3)])
@pytest.mark.parametrize("p", [0, 63, 64, 100, 149])
def test_a_large_row_does_not_reach_earlier_tokens(dtype, by, p):
    """Nor another request's, bit for bit; who sees it has it."""
    for lens, new, H, dims in SHAPES[:3]:
        s = make((150, 61), (150, 61), H=H, dims=dims, dtype=dtype)
        want = pro.check(s, "before")
        values_of(s, 0, p)[:] = by
        got = pro.check(s, f"row {p} is {by}")
        assert same(got[:p], want[:p]) and same(got[150:], want[150:])


@pytest.mark.parametrize("by", [1e30, 2.0 ** 36])
def test_another_request_does_not_reach_small_values(by):
    """Values of 1e-6 beside another request's large ones."""
    s = make((130, 61), (130, 61))
    for j in range(61):
        values_of(s, 1, j).mul_(1e-6)
    want = pro.check(s, "small")
    for j in range(130):
        values_of(s, 0, j).mul_(by)
    got = pro.check(s, f"others times {by}")
    assert same(got[130:], want[130:])


@pytest.mark.parametrize("small", [1.0, 1e-6, 1e-30])
def test_rows_without_values(small):
    """Rows whose values are all zero take part in the weights' sum alone; some tokens see nothing else."""
    s = make((200, 90, 70), (200, 90, 70), H=3)
    for b, n in ((0, 200), (1, 90), (2, 70)):
        for j in range(n):
            if j < 20 or j % 3 == 0 or b == 2:
                values_of(s, b, j).zero_()
            else:
                values_of(s, b, j).mul_(small)
    out = pro.check(s, f"zero rows beside {small}")
    assert (out[:20] == 0).all() and (out[290:] == 0).all() and (out[20:200] != 0).any()


def test_missing_pages_beside_large_rows():
    s = make((200, 90), (200, 90), H=2, extra=2)
    for j in range(0, 200, 7):
        values_of(s, 0, j).mul_(2.0 ** 50)
    s["table"][0, 3], s["table"][1, 1] = -1, s["cache"].shape[0]
    pro.check(s, "missing pages and large rows")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite_beside_large_ones(bad):
    s = make((200, 90), (200, 90), H=2)
    for j in range(0, 200, 7):
        values_of(s, 0, j).mul_(2.0 ** 50)
    want = pro.check(s, "large rows")
    values_of(s, 0, 105)[2] = bad
    got = pro.call(s)
    assert same(got[:105], want[:105]) and same(got[200:], want[200:]) and not got[105:200].isfinite().any()


def test_large_scores_beside_large_rows():
    """The row of the largest score has all the weight, whatever the sizes of the values: scores so far apart
    that float32 holds no power of two beside them.  A value is rounded once to 11 bits, the output once, and
    float32 sums over the latent dimensions are off by 2^-23 a term."""
    s = make((200,), (200,), H=2, poison=False)
    rng = np.random.default_rng(0)
    resize(s, 0, rng, -40, 40)
    s["q"].zero_()
    s["q"][..., 95] = 1.0
    s["cache"][..., s["R"]:] = 0.0
    ps, steps = s["cache"].shape[1], (0, 50, 120, 190)
    rows = s["cache"][s["table"][0].clamp(min=0).long()].reshape(-1, s["cache"].shape[2])
    for n, j in enumerate(steps):  # each above the one before it, and above the others' zero
        s["cache"][s["table"][0, j // ps].long(), j % ps, s["R"] + 31] = 2.0 ** (40 + n)
    got = f64(pro.call(s, scale=1.0))
    c, w = f64(rows[:, :s["R"]]), f64(s["w_v"])
    for t in range(200):
        j = max(x for x in steps if x <= t)
        want, size = w @ c[j], np.abs(w) @ np.abs(c[j])
        tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -3) + s["R"] * 2.0 ** -23 * size
        assert (np.abs(got[t] - want) <= tol).all(), t


def test_replays_with_rows_of_other_sizes():
    s = make((300, 90), (200, 20), H=3, poison=False)
    pro.call(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pro.call(s)
    for by in (1.0, 2.0 ** 30, 2.0 ** -30, 2.0 ** -20, 2.0 ** 70, 2.0 ** -50):
        s["cache"][..., s["half"]:s["R"]] *= by
        values_of(s, 0, 17).mul_(2.0 ** -9)
        want = pro.call(s)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), by
