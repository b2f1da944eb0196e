"""spec_tree_attention on the GPU against the float64 oracle: head layouts,
tree shapes, lengths from none to many tiles, ragged batches, windows with and
without sinks, strides, hidden rows that hold NaN, and HIP graphs."""

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import tree as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import attention_tolerance, dev, f64, parents, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def make(B=2, N=5, H=4, Hkv=2, D=64, lens=(33, 7), ps=16, kind="random", dtype=torch.bfloat16, n_nodes=None,
         head_major=False, seed=0, poison=True, extra=0):
    """Inputs on the GPU; with `poison`, rows nothing may read hold NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    pages, table = tables(lens, ps, rng, extra=extra)
    g = lambda *s: rng.standard_normal(s)  # noqa: E731
    k, v = g(pages, ps, Hkv, D), g(pages, ps, Hkv, D)
    kt, vt, q = g(B, N, Hkv, D), g(B, N, Hkv, D), g(B, N, H, D) * 2
    if poison:
        used = np.zeros((pages, ps), bool)
        for b in range(B):
            for j in range(lens[b]):
                used[table[b, j // ps], j % ps] = True
        k[~used], v[~used] = np.nan, np.nan
        if n_nodes is not None:
            for b in range(B):
                for t in (kt, vt, q):
                    t[b, max(0, n_nodes[b]):] = np.nan
    s = dict(q=dev(q, dtype), kt=dev(kt, dtype), vt=dev(vt, dtype), parent=dev(parents(kind, B, N, rng)),
             table=dev(table), lens=dev(lens), n_nodes=None if n_nodes is None else dev(np.asarray(n_nodes, np.int32)))
    for name, x in (("k", k), ("v", v)):
        s[name] = dev(x.transpose(0, 2, 1, 3), dtype).transpose(1, 2) if head_major else dev(x, dtype)
    return s


def call(s, **kw):
    return binding.tree_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["kt"], s["vt"], s["parent"],
                                  s["n_nodes"], **kw)


def oracle_of(s, **kw):
    n = None if s["n_nodes"] is None else s["n_nodes"].cpu().numpy()
    return ref.tree_attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), s["table"].cpu().numpy(), s["lens"].cpu().numpy(),
                              f64(s["kt"]), f64(s["vt"]), s["parent"].cpu().numpy(), n, **kw)


def check(s, label, **kw):
    out = call(s, **kw)
    torch.cuda.synchronize()
    want, spread, reach = oracle_of(s, **kw)
    got = f64(out)
    vmax = max(float(np.nanmax(np.abs(f64(s["v"])), initial=0.0)), float(np.nanmax(np.abs(f64(s["vt"])))))
    tol = attention_tolerance(spread, reach, want, s["q"].dtype, s["q"].shape[-1], vmax)
    seen = np.isfinite(want)  # what a node sees may be NaN (a length that reaches into unwritten slots)
    assert (np.isfinite(got) == seen).all(), label
    worst = float(np.max(np.abs(got - want)[seen] / np.maximum(tol[seen], 1e-300), initial=0.0))
    say(f"[tree attention] {label}: worst error {worst:.3f} of its bound")
    assert (np.abs(got - want)[seen] <= tol[seen]).all(), (label, worst)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hkv,N", [(4, 4, 1), (8, 2, 5), (8, 1, 9), (10, 2, 13), (16, 2, 16), (8, 2, 64), (3, 3, 33)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_and_nodes(dtype, H, Hkv, N, D):
    check(make(N=N, H=H, Hkv=Hkv, D=D, lens=(150, 61), dtype=dtype, seed=N), f"H={H} Hkv={Hkv} N={N} D={D} {dtype}")


@pytest.mark.parametrize("D", [8, 40, 72, 80, 96, 112])
def test_head_dimensions(D):
    check(make(N=6, D=D, lens=(140, 3)), f"D={D}")


@pytest.mark.parametrize("ps", [1, 2, 16, 64, 256, 1024])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths_and_pages(length, ps):
    check(make(B=1, N=4, lens=(length,), ps=ps, seed=length), f"len={length} page={ps}")


@pytest.mark.parametrize("N", [3, 12, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_long_and_ragged(N, D):
    """Lengths that differ by three orders of magnitude: parts cut across
    sequences, and single sequences over many parts."""
    lens = (2500, 0, 1, 700, 64, 1999)
    check(make(B=6, N=N, H=8, Hkv=2, D=D, lens=lens, n_nodes=[N, 0, 1, N - 1, 2, N], seed=N),
          f"ragged N={N} D={D}")


@pytest.mark.parametrize("D", [40, 80, 128])
@pytest.mark.parametrize("N,H", [(1, 1), (1, 8), (23, 5)])
def test_many_parts_of_few_sequences(N, H, D):
    """One long sequence over the whole device: its parts are joined by whole workgroups."""
    check(make(B=1, N=N, H=H, Hkv=1, D=D, lens=(9001,), ps=16, seed=N + D), f"one sequence N={N} H={H} D={D}")


def test_more_sequences_than_a_workgroup_has_threads():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 300)
    lens[250] = 900
    check(make(B=300, N=2, H=2, Hkv=1, D=64, lens=lens), "B=300")


@pytest.mark.parametrize("kind", ["chain", "star", "level2", "level3", "random"])
@pytest.mark.parametrize("N", [2, 31, 64])
def test_tree_shapes(kind, N):
    check(make(N=N, kind=kind, lens=(20, 0)), f"{kind} N={N}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (5, 0), (64, 4), (100, 130), (63, 1), (1000, 0), (128, 64)])
@pytest.mark.parametrize("N,kind", [(1, "chain"), (7, "chain"), (20, "level2")])
def test_windows(window, sinks, N, kind):
    check(make(B=3, N=N, kind=kind, D=128, lens=(700, 130, 3)), f"window={window} sinks={sinks} N={N}", window=window,
          sinks=sinks)


def test_bad_parents_end_the_line():
    s = make(B=1, N=6, lens=(9,))
    s["parent"][0] = torch.tensor([7, 5, -3, 0, 3, 1], dtype=torch.int32)  # 1: forward, 2: negative
    check(s, "bad parents")


def test_pages_outside_the_pool_are_hidden():
    s = make(B=2, N=4, lens=(100, 40), poison=True)
    s["table"][0, 2] = -1
    s["table"][0, 4] = 10 ** 6
    s["table"][1, 0] = -7
    check(s, "bad pages")
    s["lens"][0] = 10 ** 8  # clamped to the table's width: the rows behind are pages of -1
    check(s, "length beyond the table")
    s["lens"][1] = -5
    check(s, "negative length")


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_hidden_nodes_do_not_reach_others(poison):
    """A node's K and V reach its descendants only; cache rows outside a node's
    window reach the nodes that see them only."""
    s = make(B=1, N=6, kind="chain", lens=(200,), D=128, poison=False)
    s["parent"][0] = torch.tensor([-1, 0, 0, 1, 2, 0], dtype=torch.int32)
    clean = call(s)
    for name in ("kt", "vt"):
        t = make(B=1, N=6, kind="chain", lens=(200,), D=128, poison=False)
        t["parent"] = s["parent"]
        t[name][0, 2] = poison
        got = call(t)
        torch.cuda.synchronize()
        hidden = [0, 1, 3, 5]
        assert torch.equal(got[0, hidden], clean[0, hidden]), name
        if name == "vt":
            assert not torch.isfinite(got[0, [2, 4]]).any()
    # chain under a window: row len - w + 1 + d leaves the window at depth d + 1
    s = make(B=1, N=4, kind="chain", lens=(200,), D=128, poison=False)
    clean = call(s, window=50, sinks=2)
    s["v"][s["table"][0, 152 // 16].long(), 152 % 16] = poison
    got = call(s, window=50, sinks=2)
    torch.cuda.synchronize()
    assert torch.equal(got[0, 2:], clean[0, 2:])
    assert not torch.isfinite(got[0, :2]).any()


def test_visible_nan_is_not_swallowed():
    s = make(B=1, N=2, kind="chain", lens=(40,), poison=False)
    s["v"][s["table"][0, 0].long(), 3] = float("nan")
    assert torch.isnan(call(s)).all()


def test_large_scores():
    """Scores in the thousands: the running maximum carries the softmax."""
    s = make(B=2, N=8, D=128, lens=(500, 70))
    s["q"] *= 40
    check(s, "large scores")
    s = make(B=2, N=8, D=128, lens=(500, 70))
    s["q"].zero_()
    check(s, "equal scores")
    check(s, "negative scale", scale=-0.3)


@pytest.mark.parametrize("head_major", [False, True])
def test_strides(head_major):
    s = make(B=2, N=5, H=6, Hkv=2, D=80, lens=(90, 31), head_major=head_major, poison=False)
    plain = check(s, "strides")
    B, N, H, D = s["q"].shape
    packed = torch.zeros((B, N, H + 4, D), dtype=s["q"].dtype, device="cuda")
    packed[:, :, :H], packed[:, :, H:H + 2], packed[:, :, H + 2:] = s["q"], s["kt"], s["vt"]
    wide = torch.full((B, s["table"].shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"]
    s.update(q=packed[:, :, :H], kt=packed[:, :, H:H + 2], vt=packed[:, :, H + 2:],
             table=wide[:, :s["table"].shape[1]])
    room = torch.full((N, B, H, D + 8), 7.0, dtype=plain.dtype, device="cuda")
    out = room.transpose(0, 1)[..., :D]
    assert call(s, out=out) is out
    assert torch.equal(out, plain)
    assert (room[..., D:] == 7.0).all()


def test_shared_pages():
    """Two sequences whose tables name the same pages."""
    s = make(B=2, N=3, lens=(64, 50))
    s["table"][1, :4] = s["table"][0, :4]
    check(s, "shared pages")


def test_parts_do_not_change_results_between_calls():
    s = make(B=3, N=16, H=8, Hkv=2, D=128, lens=(3001, 5, 800))
    first = call(s)
    for _ in range(3):
        assert torch.equal(call(s), first)


def test_own_stream_and_two_streams_at_once():
    a, b = make(B=3, N=6, lens=(900, 20, 300), seed=1), make(B=2, N=9, lens=(1500, 70), seed=2)
    want_a, want_b = call(a), call(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        oa, ob = call(a, stream=s1), call(b, stream=s2)
        s1.synchronize()
        s2.synchronize()
        assert torch.equal(oa, want_a) and torch.equal(ob, want_b)


def test_graph_replays():
    s = make(B=3, N=6, D=128, lens=(900, 20, 300))
    other = make(B=3, N=6, D=128, lens=(900, 20, 300), seed=9)
    call(s)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(s)
    with torch.cuda.graph(second):
        out2 = call(other)
    for rep in range(4):
        n = make(B=3, N=6, D=128, lens=(900 - rep, 20 + rep, 300), seed=10 + rep)
        s["lens"].copy_(n["lens"])
        s["q"].copy_(n["q"])
        want = call(s)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        # bit for bit: the longer length reaches a slot that was never written (NaN)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), rep
        assert torch.equal(out2, call(other)), rep


@pytest.mark.parametrize("name", ["k", "v", "kt", "vt"])
@pytest.mark.parametrize("lens", [(100, 40), (9000, 40)])  # one part each; the first divided
@pytest.mark.parametrize("N,H", [(6, 4), (20, 4), (40, 6)])  # rows that fill 32, 64 and more than 64
def test_absent_nodes_stay_zero_beside_visible_nan(N, H, lens, name):
    """An absent node's row is zero whatever the rows hold that others see."""
    for bad in (float("nan"), float("inf")):
        s = make(B=2, N=N, H=H, kind="chain", lens=lens, n_nodes=[2, 3], poison=False, seed=N)
        for b in range(2):
            if name in ("k", "v"):
                s[name][s["table"][b, 0].long(), 3] = bad
            else:
                s[name][b, 0] = bad
        out = call(s)
        torch.cuda.synchronize()
        for b, n in enumerate((2, 3)):
            assert (out[b, n:] == 0).all(), (b, bad)
            assert not torch.isfinite(out[b, 0]).any(), (b, bad)


@pytest.mark.parametrize("bits", [21.6, 25.5])
@pytest.mark.parametrize("N,H", [(2, 8), (8, 8), (16, 8)])  # 16, 64 and 128 rows per key head
def test_float16_tail_behind_a_dominant_key(N, H, bits):
    """One key (an attention sink) `bits` powers of two above 32767 equal ones:
    their weights are far below float16's normal numbers next to its own.  As
    many (sequence, key head)s as the device has parts, so that none is divided
    and the tail meets the sink's maximum; all sequences share their pages.

    Bound: attention_tolerance's with its absolute term at 2^-32 a key.  Weights
    are held times 2^7, so half the spacing of float16's subnormals, 2^-25, is
    2^-32 of the row's reference (parts' and waves' own references are below the
    row's, and their errors shrink with them)."""
    B, Hkv, D, ps, n = 512, 1, 64, 1024, 32768
    rng = np.random.default_rng(1)
    k, v = np.zeros((n // ps, ps, Hkv, D)), 1 + 0.25 * rng.random((n // ps, ps, Hkv, D))
    k[0, 0, 0, 0], v[0, 0] = bits * np.log(2), 0.0
    q, kt, vt = np.zeros((1, N, H, D)), np.zeros((1, N, Hkv, D)), 1 + 0.25 * rng.random((1, N, Hkv, D))
    q[..., 0] = 1.0
    table = np.arange(n // ps, dtype=np.int32)[None]
    par = parents("chain", 1, N, rng)
    all_of = lambda a, dtype=None: dev(np.repeat(a, B, 0), dtype)  # noqa: E731
    f16 = torch.float16
    s = dict(q=all_of(q, f16), kt=all_of(kt, f16), vt=all_of(vt, f16), parent=all_of(par), table=all_of(table),
             lens=dev(np.full(B, n, np.int32)), n_nodes=None, k=dev(k, f16), v=dev(v, f16))
    out = call(s, scale=1.0)
    torch.cuda.synchronize()
    assert (out == out[:1]).all()
    want, spread, reach = ref.tree_attention(f64(s["q"][:1]), f64(s["k"]), f64(s["v"]), table, np.array([n]),
                                             f64(s["kt"][:1]), f64(s["vt"][:1]), par, scale=1.0)
    vmax = 1.25
    tol = attention_tolerance(spread, reach, want, f16, D, 0.0) + reach[..., 1:2] * 2.0 ** -32 * vmax
    worst = float((np.abs(f64(out[:1]) - want) / tol).max())
    say(f"[tree attention] {bits} bits, {N * H} rows: output {want.max():.2e}, worst error {worst:.3f} of its bound")
    assert worst <= 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,H", [(4, 4), (20, 4), (40, 6)])
def test_visible_nan_of_vanishing_weight_is_not_swallowed(N, H, bad):
    """A node that sees a NaN or infinite value gives no finite number, also
    where the key's weight is below float32's smallest: in the tree, and in a
    tile of which the window hides rows from some nodes."""
    s = make(B=1, N=N, H=H, kind="chain", lens=(200,), poison=False)
    D = s["q"].shape[-1]
    s["q"][0, 2], s["kt"][0, 0], s["vt"][0, 0] = 8.0, -8.0, bad  # a score of -512 beside ones of size 10
    out = call(s)
    torch.cuda.synchronize()
    assert not torch.isfinite(out).any()
    s = make(B=1, N=N, H=H, kind="chain", lens=(200,), poison=False)
    pg, slot = s["table"][0, 152 // 16].long(), 152 % 16  # the root and its child see row 152, the others do not
    s["q"][0, 1], s["k"][pg, slot], s["v"][pg, slot] = 8.0, -8.0, bad
    out = call(s, window=50)
    torch.cuda.synchronize()
    assert D == 64 and not torch.isfinite(out[0, :2]).any() and torch.isfinite(out[0, 2:]).all()


def test_tables_of_ever_new_widths_keep_a_bounded_record():
    """A decoder that sizes its tables to the batch: the kept workspace sizes
    do not grow with it."""
    s = make(B=1, N=1, lens=(5,))
    wide = torch.full((1, 1200), -1, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"]
    for w in range(1, 1201):
        s["table"] = wide[:, :w]
        call(s)
    torch.cuda.synchronize()
    assert len(binding._workspaces) <= 1024
    check(s, "1200 pages wide")


@pytest.mark.parametrize("dtype,size,far", [(torch.bfloat16, 60, 4), (torch.bfloat16, 30, 10), (torch.bfloat16, 8, 8),
                                            (torch.float16, 15, 14), (torch.float16, 12, 11), (torch.float16, 8, 4)])
@pytest.mark.parametrize("N,H", [(2, 8), (8, 8), (16, 8)])  # 16, 64 and 128 rows per key head
@pytest.mark.parametrize("lens", [(190,), (3001,)])
def test_scores_beyond_the_float32_spacing(lens, N, H, dtype, size, far):
    """Scores so large that float32 keeps no fraction of them: the key of the
    largest one (its neighbours in the input type are far below it) has all the
    weight, and its value is the output, exactly."""
    s = make(B=1, N=N, H=H, Hkv=1, kind="chain", lens=lens, dtype=dtype, poison=False)
    rng = np.random.default_rng(3)
    n, D = lens[0], s["q"].shape[-1]
    for name in ("q", "k", "kt"):
        s[name].zero_()
    s["q"][..., 0] = 2.0 ** size
    x = rng.permutation(n)  # one key of 3.5 * 2^far, the others from 1 to 2 times that power
    pages, slots = s["table"][0, np.arange(n) // 16].long(), torch.from_numpy(np.arange(n) % 16).cuda()
    s["k"][pages, slots, 0, 0] = dev(np.where(x == 0, 3.5, 1 + x / n) * 2.0 ** far, dtype)
    top = int((x == 0).argmax())
    s["q"][0, 1:, :, 0] *= -1  # for the other nodes the root's, the only one below zero
    s["kt"][0, :, 0, 0] = 8.0
    s["kt"][0, 0, 0, 0] = -8.0
    out = call(s, scale=0.3)
    torch.cuda.synchronize()
    root = s["v"][pages[top], slots[top], 0]
    assert torch.equal(out[0, 0], root.expand(H, D))
    assert torch.equal(out[0, 1:], s["vt"][0, 0, 0].expand(N - 1, H, D))


def test_largest_batches_and_row_counts():
    """The limits the header states: 65536 sequences, 65536 query rows per key
    head, an empty table, windows and sinks up to 2^31 - 1."""
    B = 65536
    for width in (1, 300):  # whole parts, and parts over several sequences
        s = make(B=2, N=1, H=2, Hkv=1, D=8, lens=(9, 16), ps=16, poison=False)
        lens = torch.arange(B, dtype=torch.int32, device="cuda") % 17
        q = torch.randn((B, 1, 2, 8), device="cuda").bfloat16()
        kt, vt = torch.randn((B, 1, 1, 8), device="cuda").bfloat16(), torch.randn((B, 1, 1, 8), device="cuda").bfloat16()
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = torch.arange(B, device="cuda") % s["k"].shape[0]
        out = binding.tree_attention(q, s["k"], s["v"], table, lens, kt, vt,
                                     torch.full((B, 1), -1, dtype=torch.int32, device="cuda"))
        kk = torch.cat((s["k"][table[:, 0].long(), :, 0], kt[:, :, 0]), 1).double()
        vv = torch.cat((s["v"][table[:, 0].long(), :, 0], vt[:, :, 0]), 1).double()
        x = (kk.unsqueeze(1) * q[:, 0].double().unsqueeze(2)).sum(-1) * 8 ** -0.5  # [B, heads, 17]
        j = torch.arange(17, device="cuda")
        x = torch.where((j < lens.view(B, 1, 1)) | (j == 16), x, -torch.inf)
        w = torch.softmax(x, -1)
        want = (w.unsqueeze(-1) * vv.unsqueeze(1)).sum(2)
        spread = (w.unsqueeze(-1) * vv.abs().unsqueeze(1)).sum(2)
        tol = 2.0 ** -8 * (spread + want.abs()) * 1.01 + 1e-30  # two roundings; float32's are 2^-14 of them
        assert ((out[:, 0].double() - want).abs() <= tol).all(), width
    s = make(B=1, N=64, H=1024, Hkv=1, D=8, lens=(70,), ps=16)
    check(s, "65536 rows")
    s = make(B=3, N=5, lens=(0, 0, 0))
    s["table"] = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    check(s, "an empty table")
    s = make(B=2, N=5, lens=(200, 40))
    plain = call(s)
    big = 2 ** 31 - 1
    for kw in (dict(window=big), dict(window=big, sinks=big), dict(window=1, sinks=big)):
        out = call(s, **kw)
        torch.cuda.synchronize()
        if kw["window"] == big:
            assert torch.equal(out, plain)
        else:
            check(s, "all sinks", **kw)


def test_expanded_inputs():
    """One set of rows for all sequences and one key head for all."""
    s = make(B=3, N=4, H=4, Hkv=2, D=64, lens=(50, 9, 31), poison=False)
    e = dict(s, q=s["q"][:1].expand(3, -1, -1, -1), kt=s["kt"][:, :, :1].expand(-1, -1, 2, -1),
             vt=s["vt"][:, :1].expand(-1, 4, -1, -1), k=s["k"][:, :, :1].expand(-1, -1, 2, -1),
             table=s["table"][:1].expand(3, -1))
    got = check(e, "expanded")
    whole = {n: (t.contiguous() if t is not None else None) for n, t in e.items()}
    assert torch.equal(call(whole), got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H", [(1, 1), (8, 8), (16, 8)])
def test_the_longest_cache(N, H, dtype):
    """2^28 cache rows: a table of 2^18 pages that are all one of two, so that
    the softmax is that of two pages, each key 2^17 times.

    The sums are float32: a wave adds its weights key by key (32 lanes' worth at
    a time), up to 2^28 / 512 parts / 4 keys of one row, each rounding at most
    2^-24 of the running sum, and the matrix unit's sums 2^-23; relative to
    sums of positive terms 2^17 * 2^-23 at worst, where roundings do not cancel.
    They do: 2^-9 (their square root times 2^-1) is allowed beside the roundings
    to the input type."""
    D, ps, width = 64, 1024, 1 << 18
    s = make(B=1, N=N, H=H, Hkv=1, D=D, kind="chain", lens=(2 * ps,), ps=ps, dtype=dtype, poison=False)
    two = s["table"][0, :2].clone()
    s["table"] = two.repeat(width // 2).view(1, width).contiguous()
    s["lens"].fill_(1 << 28)
    out = call(s)
    torch.cuda.synchronize()
    k = torch.cat((s["k"][two.long()].reshape(-1, D), s["kt"][0, :, 0])).double()
    v = torch.cat((s["v"][two.long()].reshape(-1, D), s["vt"][0, :, 0])).double()
    x = (s["q"][0].double().reshape(-1, D).mm(k.t().contiguous()) * D ** -0.5).view(N, H, -1)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w[..., :2 * ps] *= width // 2
    w[..., 2 * ps:] *= (torch.arange(N, device="cuda").view(1, N) <= torch.arange(N, device="cuda").view(N, 1)).unsqueeze(1)
    w /= w.sum(-1, keepdim=True)
    want, spread = (w.view(N * H, -1).mm(t) for t in (v, v.abs()))
    err = (out[0].double().view(N * H, D) - want).abs()
    h = torch.finfo(dtype).eps / 2
    assert (err <= (h + 2.0 ** -9) * spread + h * want.abs() + 1e-6).all(), float((err / spread).max())
    # a window of all but the first rows, and of a few rows at the end
    for window in ((1 << 28) - 100, 3000):
        part = call(s, window=window, sinks=5)
        torch.cuda.synchronize()
        assert torch.isfinite(part).all()
    near = dict(s, table=s["table"][:, :4].contiguous(), lens=torch.full((1,), 4 * ps, dtype=torch.int32, device="cuda"))
    a, b = call(s, window=3000), call(near, window=3000)
    torch.cuda.synchronize()
    assert ((a.double() - b.double()).abs() <= 4 * h * spread.amax().item()).all()


@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.4e38])
def test_scales_near_the_largest_float(scale):
    """scale log2(e) lies beyond float32 there: equal scores stay equal, and the
    key of the largest score has all the weight."""
    s = make(B=1, N=3, kind="chain", lens=(40,), poison=False)
    for name in ("q", "k", "kt"):
        s[name].zero_()
    check(s, f"scale {scale}", scale=scale)
    s["q"][..., 0] = 1.0 if scale > 0 else -1.0
    page = s["table"][0, 1].long()
    s["k"][page, 3, :, 0] = 2.0 ** -30
    out = call(s, scale=scale)
    torch.cuda.synchronize()
    want = s["v"][page, 3].repeat_interleave(2, 0)
    assert torch.equal(out[0], want.expand(3, -1, -1))
