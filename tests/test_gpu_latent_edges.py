"""Where the calls on latent rows can go wrong: NaN and infinities in rows that
are hidden or seen, pages outside the pool, lengths and bounds out of range,
extreme scales and magnitudes, strides, offsets past 32 bits, used workspaces,
other streams, two calls at once, HIP graphs."""

import numpy as np
import pytest
import torch

import test_gpu_latent_attention as att
import test_gpu_latent_prompt as pro
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def same(a, b):
    """Equal bit for bit, NaN included."""
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def at(s, b, j):
    """Row j of sequence b in its cache."""
    ps = s["cache"].shape[1]
    return s["cache"][s["table"][b, j // ps].long(), j % ps]


# ---- attention on the rows

@pytest.mark.parametrize("poison", [NAN, INF, -INF])
@pytest.mark.parametrize("N,H", [(6, 4), (20, 3), (12, 16)])  # rows that fill 32, 64 and more than 64
def test_hidden_nodes_do_not_reach_others(poison, N, H):
    """Node 1 is on nobody's path but its own."""
    s = att.make(N=N, H=H, lens=(130, 0))
    s["parent"][:, 1] = 0
    s["parent"][:, 2:][s["parent"][:, 2:] == 1] = 0
    want = att.call(s)
    s["rows"][:, 1] = poison
    got = att.call(s)
    keep = [i for i in range(N) if i != 1]
    assert same(got[:, keep], want[:, keep]) and got[:, 1].isnan().all()


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("N,H", [(4, 4), (20, 3), (12, 16)])
@pytest.mark.parametrize("where", [0, 511, 512])  # of the values, and the first that is a key's only
def test_visible_rows_that_are_not_finite(bad, N, H, where):
    """A chain: the node and those behind it; a cache row: the whole sequence.
    The infinity meets a positive element of the queries: a score of +inf."""
    s = att.make(N=N, H=H, lens=(100, 40), kind="chain")
    s["q"][..., where] = 1.0
    want = att.call(s)
    s["rows"][0, 2, where] = bad
    got = att.call(s)
    assert same(got[1], want[1]) and same(got[0, :2], want[0, :2]) and got[0, 2:].isnan().all()
    s["rows"][0, 2, where] = 0.0
    at(s, 0, 77)[where] = bad
    got = att.call(s)
    assert same(got[1], want[1]) and got[0].isnan().all()


@pytest.mark.parametrize("bad", [NAN, INF])
def test_visible_node_of_vanishing_weight_is_not_swallowed(bad):
    s = att.make(B=1, N=3, H=4, lens=(60,), kind="chain", poison=False)
    s["q"].zero_()
    s["q"][..., 575] = 1.0
    s["cache"][..., 575] = 0.0
    s["rows"][..., 575] = -30000.0  # exp(-30000 / 24) is no float
    s["rows"][0, 1, 3] = bad
    got = att.call(s)
    assert got[0, 0].isfinite().all() and got[0, 1:, :, 3].isnan().all()


def test_pages_outside_the_pool_are_left_out():
    s = att.make(B=3, N=4, H=5, lens=(200, 90, 40), extra=2)
    pages = s["cache"].shape[0]
    s["table"][0, 3], s["table"][0, 7], s["table"][1, 0] = -1, pages, 2 ** 31 - 1
    s["table"][2, :] = -2 ** 31
    att.check(s, "missing pages")


@pytest.mark.parametrize("N,H", [(3, 4), (9, 16)])
def test_lengths_and_counts_out_of_range(N, H):
    """Clipped to what the table holds and to [0, N]."""
    s = att.make(B=4, N=N, H=H, lens=(50, 16, 33, 20), poison=False, n_nodes=[N + 9, -4, 2 ** 31 - 1, 1])
    s["table"].clamp_(0)
    s["lens"].copy_(dev(np.array([2 ** 31 - 1, -1, -2 ** 31, 64], np.int32)))
    att.check(s, "out of range")


def test_no_cache_at_all():
    s = att.make(B=2, N=5, H=4, lens=(0, 0), kind="random")
    full = att.check(s, "no rows")
    s["table"] = s["table"][:, :0]
    assert same(att.call(s), full)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(scale):
    s = att.make(B=2, N=4, H=6, lens=(140, 9), gain=0.5)
    s["scale"] = scale
    att.check(s, f"scale {scale}")


@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.4e38])
def test_scales_near_the_largest_float(scale):
    """scale log2(e) lies beyond float32 there: equal scores stay equal, and the
    row of the largest score has all the weight."""
    s = att.make(B=1, N=3, H=4, kind="chain", lens=(40,), poison=False)
    s["q"].zero_()
    s["scale"] = scale
    att.check(s, f"scale {scale}")
    s["q"][..., 575] = 1.0 if scale > 0 else -1.0
    for t in (s["cache"], s["rows"]):
        t[..., 575] = 0.0
    row = at(s, 0, 19)
    row[575] = 2.0 ** -30
    assert torch.equal(att.call(s)[0], row[:512].expand(3, 4, 512))


def test_scores_that_rise_along_the_cache():
    """The running maximum is raised again and again, by little and by much."""
    s = att.make(B=2, N=2, H=20, lens=(1500, 700), gain=1.0)
    for b, n in ((0, 1500), (1, 700)):
        for j in range(0, n, 37):
            at(s, b, j)[570] = j / 8.0
    s["q"][..., 570] = 1.5
    s["q"][:, :, ::2, 570] = -0.3
    att.check(s, "rising scores")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("C,dv", [(576, 512), (288, 256)])
def test_strides(dtype, C, dv):
    """Heads before nodes, a layer of a cache with slots before pages, slices of
    wider rows; what lies around the output stays."""
    s = att.make(B=2, N=5, H=6, C=C, dv=dv, lens=(90, 31), dtype=dtype)
    want = att.check(s, "plain")
    q, cache, rows = s["q"], s["cache"], s["rows"]
    wide = torch.full((2, 6, 5, C + 24), NAN, dtype=dtype, device="cuda").transpose(1, 2)[..., 8:8 + C]
    wide.copy_(q)
    pool = torch.full((16, cache.shape[0], 3, C), NAN, dtype=dtype, device="cuda")[:, :, 1].transpose(0, 1)
    pool.copy_(cache)
    node = torch.full((5, 2, C + 8), NAN, dtype=dtype, device="cuda").transpose(0, 1)[..., :C]
    node.copy_(rows)
    tab = torch.full((2, s["table"].shape[1] + 3), 10 ** 6, dtype=torch.int32, device="cuda")[:, 1:-2]
    tab.copy_(s["table"])
    full = torch.full((5, 2, 8, dv + 16), -7.0, dtype=dtype, device="cuda")
    out = full[:, :, 1:7, 8:8 + dv].transpose(0, 1)
    s.update(q=wide, cache=pool, rows=node, table=tab)
    assert att.call(s, out=out) is out and same(out, want)
    full[:, :, 1:7, 8:8 + dv] = -7.0
    assert (full == -7.0).all()


def test_expanded_inputs_and_shared_pages():
    s = att.make(B=3, N=4, H=4, lens=(60, 60, 60), kind="chain", poison=False)
    s["table"][1:] = s["table"][0]
    s["q"] = s["q"][:1, :, :1].expand(3, 4, 4, 576)
    s["rows"] = s["rows"][:1].expand(3, 4, 576)
    out = att.check(s, "expanded")
    assert same(out[0], out[2]) and same(out[:, :, 0], out[:, :, 3])


def test_most_rows():
    att.check(att.make(B=1, N=64, H=1024, C=64, dv=8, lens=(70,)), "65536 rows")


def test_largest_batch():
    rng = np.random.default_rng(0)
    att.check(att.make(B=65536, N=1, H=1, C=16, dv=8, lens=rng.integers(0, 4, 65536), ps=4), "65536 sequences")


def test_offsets_past_32_bits():
    """Rows 5 GB into the cache, bit for bit as from a small one."""
    s = att.make(B=2, N=3, H=16, lens=(300, 90), poison=False)
    want = att.call(s)
    pages = 300000
    big = torch.empty((pages, 16, 576), dtype=BF16, device="cuda")
    used = s["cache"].shape[0]
    big[-used:] = s["cache"]
    live = s["table"] >= 0
    s["table"][live] += pages - used
    s["cache"] = big
    assert same(att.call(s), want)


def test_calls_do_not_change_results():
    s = att.make(B=3, N=16, H=8, lens=(3001, 5, 800))
    first = att.call(s)
    for junk in (0xFF, 0x00, 0x7F):
        need = 64 << 20
        torch.full((need,), junk, dtype=torch.uint8, device="cuda")  # freed: the next workspace lies in it
        assert same(att.call(s), first)


def test_own_stream_and_two_streams_at_once():
    a, b = att.make(B=3, N=6, lens=(900, 20, 300), seed=1), att.make(B=2, N=9, lens=(1500, 70), seed=2)
    c = pro.make((300, 40), (300, 7), H=4)
    wants = att.call(a), att.call(b), pro.call(c)
    torch.cuda.synchronize()
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    for _ in range(6):
        outs = att.call(a, stream=s1), att.call(b, stream=s2), pro.call(c, stream=s3)
        for x in (s1, s2, s3):
            x.synchronize()
        assert all(same(x, y) for x, y in zip(outs, wants))


def test_attention_graph_replays():
    s = att.make(B=3, N=6, lens=(900, 20, 300), poison=False)
    other = att.make(B=3, N=6, lens=(900, 20, 300), seed=9)
    att.call(s)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = att.call(s)
    with torch.cuda.graph(second):
        out2 = att.call(other)
    for rep in range(4):
        s["lens"].copy_(dev(np.array([900 - 300 * rep, 20 + rep, 300], np.int32)))
        s["q"].mul_(0.5)
        want = att.call(s)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        assert same(out, want) and same(out2, att.call(other)), rep


# ---- products

@pytest.mark.parametrize("T", [9, 200])
def test_product_rows_keep_to_themselves(T):
    x, w = pro.operands(T, 3, 72, 136, BF16)
    want = binding.head_product(x, w)
    x[2, 1, 5], x[3, 0] = NAN, INF
    got = binding.head_product(x, w)
    assert got[2, 1].isnan().all() and not got[3, 0].isfinite().any()
    clean = torch.ones((T, 3), dtype=torch.bool, device="cuda")
    clean[2, 1] = clean[3, 0] = False
    assert same(got[clean], want[clean])


def test_product_stream_and_graph():
    x, w = pro.operands(150, 3, 72, 136, BF16)
    want = binding.head_product(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = binding.head_product(x, w, stream=side)
    side.synchronize()
    assert same(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.head_product(x, w)
    for rep in range(3):
        x.neg_()
        want = binding.head_product(x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), rep


# ---- prompts

@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("p", [0, 63, 64, 100, 149])
def test_later_rows_do_not_reach_earlier_tokens(bad, p):
    s = pro.make((150, 61), (150, 20), H=2, dims=(64, 32, 64, 128))
    at(s, 0, p)[3] = bad
    out = pro.check(s, f"row {p} is {bad}")
    assert out[:p].isfinite().all() and not out[p:150].isfinite().any() and out[150:].isfinite().all()


@pytest.mark.parametrize("row", [0, 5, 60, 70])
def test_value_beyond_float32_of_one_row(row):
    """A row whose keys are finite and one of whose values is not: every token that
    sees it, wherever it lies in a tile of queries."""
    s = pro.make((200,), (200,), H=2, dims=(64, 32, 64, 128), poison=False)
    s["cache"][..., 7] = 0.0
    s["w_k"][:, :, 7] = 0.0
    s["w_v"][:, :, 7] = 0.0
    s["w_v"][1, 3, 7] = 3e38
    want = pro.call(s)
    at(s, 0, row)[7] = 3e38
    out = pro.call(s)
    assert same(out[:, 0], want[:, 0]) and same(out[:row], want[:row])
    assert not out[row:, 1, 3].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_many_heads_on_many_rows(dtype):
    """Keys and values of 130 heads for 2200 rows: more large tiles than the device holds twice."""
    s = pro.make((700, 3, 1497), (9, 3, 5), H=130, dims=(64, 32, 72, 136), dtype=dtype)
    s["w_v"][7] *= 1e-3
    pro.check(s, f"130 heads {dtype}")


def test_missing_pages_of_prompts():
    s = pro.make((200, 90, 40), (200, 30, 40), H=2, dims=(64, 32, 64, 128), extra=2)
    pages = s["cache"].shape[0]
    s["table"][0, 0], s["table"][0, 7], s["table"][1, 1] = -1, pages, 2 ** 31 - 1
    s["table"][2, :] = -2 ** 31
    out = pro.check(s, "missing pages")
    assert (out[230:] == 0).all()


def test_prompt_lengths_out_of_range():
    s = pro.make((50, 16, 33, 64), (20, 5, 7, 3), H=2, dims=(64, 32, 64, 128), poison=False)
    s["table"].clamp_(0)
    s["lens"].copy_(dev(np.array([2 ** 31 - 1, -1, -2 ** 31, 64], np.int32)))
    s["rows"] = 400
    pro.check(s, "lengths out of range")


def test_rows_that_do_not_fit():
    """The bound is too small by one: the last sequence is NaN, the others as before."""
    s = pro.make((70, 300, 41), (70, 100, 41), H=2, dims=(64, 32, 64, 128))
    want = pro.check(s, "all fit")
    out = pro.call(s, rows=s["rows"] - 1)
    assert same(out[:170], want[:170]) and out[170:].isnan().all()
    assert pro.call(s, rows=0).isnan().all()
    assert same(pro.call(s, rows=s["rows"] + 1000), want)


def test_queries_without_rows_behind_a_line_that_is_full():
    s = pro.make((70, 0), (70, 4), H=2, dims=(64, 32, 64, 128))
    out = pro.call(s, rows=60)
    assert out[:70].isnan().all() and (out[70:] == 0).all()


def test_rows_of_no_sequence_stay():
    s = pro.make((70, 30, 41), (60, 30, 11), H=2, dims=(64, 32, 64, 128), poison=False)
    want = pro.call(s)
    s["q"] = torch.cat((s["q"].new_full((3, 2, 96), NAN), s["q"], s["q"].new_full((9, 2, 96), NAN)))
    s["start"] += 3
    out = torch.full((113, 2, 64), -7.0, dtype=BF16, device="cuda")
    pro.call(s, out=out)
    assert same(out[3:104], want) and (out[:3] == -7.0).all() and (out[104:] == -7.0).all()
    for start, mine in (((3, 63, 20, 104), (3, 63)), ((-5, 63, 93, 104), (63, 104)), ((3, 63, 93, 400), (3, 93)),
                        ((9, 9, 9, 9), (0, 0))):
        out.fill_(-7.0)
        s["start"].copy_(dev(np.array(start, np.int32)))
        pro.call(s, out=out)
        lo, hi = mine
        assert (out[:lo] == -7.0).all() and out[lo:hi].isfinite().all(), start
        seen = torch.zeros(113, dtype=torch.bool, device="cuda")
        for a, e in zip(start, start[1:]):
            if 0 <= a < e <= 113:
                seen[a:e] = True
        assert (out[~seen] == -7.0).all(), start


@pytest.mark.parametrize("dtype,by", [(BF16, 1e30), (BF16, 1e5), (BF16, 1e-6), (BF16, 1e-30), (FP16, 300.0), (FP16, 1e-3)])
def test_magnitudes_of_values(dtype, by):
    """Values beyond float16's range and below its smallest: a power of two per head keeps them."""
    s = pro.make((150, 61), (150, 20), H=3, dims=(64, 32, 64, 128), dtype=dtype)
    s["w_v"][1] *= by
    pro.check(s, f"values times {by}")


def test_one_head_without_values():
    s = pro.make((150,), (150,), H=3, dims=(64, 32, 64, 128))
    s["w_v"][1] = 0.0
    assert (pro.check(s, "zero values")[:, 1] == 0).all()


@pytest.mark.parametrize("scale", [3.4e38, -3.4e38])
def test_prompt_scales_near_the_largest_float(scale):
    s = pro.make((60,), (60,), H=2, dims=(8, 8, 64, 64), poison=False)
    s["q"].zero_()
    pro.check(s, f"scale {scale}", scale=scale)
    s["q"][..., 15] = 1.0 if scale > 0 else -1.0
    s["cache"][..., 71] = 0.0
    at(s, 0, 5)[71] = 2.0 ** -30
    out = pro.call(s, scale=scale)
    assert out.isfinite().all() and same(out[5:], out[5:6].expand(55, 2, 64))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_prompt_strides(dtype):
    s = pro.make((90, 31), (50, 31), H=4, dims=(64, 32, 72, 128), dtype=dtype)
    want = pro.check(s, "plain")
    q, cache = s["q"], s["cache"]
    wide = torch.full((4, 81, 120), NAN, dtype=dtype, device="cuda").transpose(0, 1)[..., 16:112]
    wide.copy_(q)
    pool = torch.full((16, cache.shape[0], 2, 160), NAN, dtype=dtype, device="cuda")[:, :, 1].transpose(0, 1)
    pool.copy_(cache)
    both = torch.full((4, 136, 136), NAN, dtype=dtype, device="cuda")
    both[:, :64, :128], both[:, 64:, :128] = s["w_k"], s["w_v"]
    full = torch.full((6, 81, 88), -7.0, dtype=dtype, device="cuda")
    out = full[1:5, :, 8:80].transpose(0, 1)
    s.update(q=wide, cache=pool, w_k=both[:, :64, :128], w_v=both[:, 64:, :128])
    assert pro.call(s, out=out) is out and same(out, want)
    full[1:5, :, 8:80] = -7.0
    assert (full == -7.0).all()


def test_prompt_offsets_past_32_bits():
    s = pro.make((300, 90), (300, 20), H=2, dims=(64, 64, 64, 512), poison=False)
    want = pro.call(s)
    pages, used = 300000, s["cache"].shape[0]
    big = torch.empty((pages, 16, 576), dtype=BF16, device="cuda")
    big[-used:] = s["cache"]
    s["table"][s["table"] >= 0] += pages - used
    s["cache"] = big
    assert same(pro.call(s), want)


def test_prompt_of_no_tokens_and_used_workspaces():
    s = pro.make((30, 20), (0, 0), H=2, dims=(64, 32, 64, 128))
    assert pro.call(s).shape == (0, 2, 64)
    s = pro.make((300, 65), (130, 65), H=3)
    first = pro.call(s)
    for junk in (0xFF, 0x00, 0x7F):
        torch.full((64 << 20,), junk, dtype=torch.uint8, device="cuda")  # freed: the next workspace lies in it
        assert same(pro.call(s), first)


def test_prompt_graph_replays():
    s = pro.make((300, 90), (200, 20), H=3, poison=False)
    other = pro.make((130, 9), (130, 9), H=2, seed=7)
    pro.call(s)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pro.call(s)
    with torch.cuda.graph(second):
        out2 = pro.call(other)
    for rep in range(4):
        s["lens"].copy_(dev(np.array([300 - 30 * rep, 90], np.int32)))
        s["q"].mul_(0.7)
        s["w_v"].mul_(40.0)  # the values' power of two is found anew by every replay
        want = pro.call(s)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        assert same(out, want) and same(out2, pro.call(other)), rep


# ---- beams and reservations

def test_beam_stream_and_graph():
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn((3, 8, 20011), generator=g, device="cuda") * 3
    scores = -torch.rand((3, 8), generator=g, device="cuda").sort(-1)[0]
    done = torch.zeros((3, 8), dtype=torch.int32, device="cuda")
    state = torch.randint(0, 9, (24, 37), generator=g, device="cuda", dtype=torch.int32)

    def run(**kw):
        picked = binding.beam_select(logits, scores, done, end=5, **kw)
        return (*picked, binding.beam_reorder(state, picked[1], **kw))

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for rep in range(4):
        logits.copy_(logits.roll(101, -1) * 0.9)
        scores[:, rep] = -INF
        done[0, 7 - rep] = 1
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep


def test_reserve_stream_and_graph():
    rng = np.random.default_rng(0)
    table = torch.full((5, 60), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(5, dtype=torch.int32, device="cuda")
    new = dev(np.array([100, 0, 33, 16, 1], np.int32))
    cache = torch.zeros((300, 16, 40), dtype=BF16, device="cuda")
    x = dev(rng.standard_normal((200, 40)), BF16)

    def run(**kw):
        got = binding.cache_reserve(table, lens, new, pages=300, page_size=16, rows=200, **kw)
        binding.cache_write(cache, got[3], x[:, :32], x[:, 32:], **kw)
        return got

    want, filled = run(), cache.clone()
    cache.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(cache, filled)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for rep in range(4):
        table.copy_(want[0])
        lens.copy_(want[1])
        new.copy_(dev(rng.integers(0, 40, 5).astype(np.int32)))
        before = cache.clone()
        want, filled = run(), cache.clone()
        cache.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(cache, filled), rep


def test_a_write_past_32_bits():
    cache = torch.zeros((300000, 16, 576), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((40, 576), generator=g, device="cuda").to(BF16)
    slots = torch.arange(300000 * 16 - 40, 300000 * 16, dtype=torch.int32, device="cuda")
    binding.cache_write(cache, slots, x[:, :512], x[:, 512:])
    assert torch.equal(cache.view(-1, 576)[-40:], x) and (cache.view(-1, 576)[:-40] == 0).all()


def test_logits_past_32_bits():
    """A batch of 6 GB: the last sequence as it is alone."""
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.zeros((90, 16, 1 << 20), dtype=torch.float32, device="cuda")
    logits[-1].normal_(generator=g)
    scores = -torch.rand((90, 16), generator=g, device="cuda")
    got, alone = binding.beam_select(logits, scores), binding.beam_select(logits[-1:].clone(), scores[-1:].clone())
    assert torch.equal(got[0][-1:], alone[0]) and torch.equal(got[2][-1:], alone[2])
    assert torch.equal(got[1][-16:] - 89 * 16, alone[1])
