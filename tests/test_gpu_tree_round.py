"""The tree round's calls one after another, as a decoder runs them: a small
random transformer drafts trees (or chains, or particles), attends over its
paged cache, verifies and commits for several rounds.  Every call is compared
with the oracle on the inputs it had, and at the end the cache must hold, page
by page, the rows of the tokens that were accepted and nothing of the others."""

import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import tree as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import attention_tolerance, dev, f64, parents

pytestmark = pytest.mark.gpu

L, H, HKV, D, V, PS = 2, 8, 2, 64, 997, 8  # layers, heads, key heads, dimension, vocabulary, page size
PAGES, WIDTH = 60, 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


class Model:
    """Layer 0's keys and values depend on the token alone, so that what the
    cache must hold there is known without the model."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, by=1.0: (torch.randn(s, generator=g, device="cuda") * by)  # noqa: E731
        E = 96
        self.emb = r(V, E)
        self.wq = [r(E, H * D, by=E ** -0.5) for _ in range(L)]
        self.wk = [r(E, HKV * D, by=E ** -0.5) for _ in range(L)]
        self.wv = [r(E, HKV * D, by=E ** -0.5) for _ in range(L)]
        self.wo = [r(H * D, E, by=(H * D) ** -0.5) for _ in range(L)]
        self.head = r(E, V, by=2 * E ** -0.5)
        self.draft_head = self.head + r(E, V, by=0.5 * E ** -0.5)
        first = (self.emb @ self.wk[0]).bfloat16(), (self.emb @ self.wv[0]).bfloat16()
        self.k0, self.v0 = (t.view(V, HKV, D) for t in first)

    def draft(self, tokens):
        """The draft's distribution after each token: [.., V] float32."""
        return torch.softmax(self.emb[tokens.long()] @ self.draft_head, -1)

    def forward(self, s, tok, par, n_nodes=None, attend=None):
        """Target probabilities after every node, and the nodes' rows."""
        B, N = tok.shape
        x = self.emb[tok.long()]
        kt = torch.empty((L, B, N, HKV, D), dtype=torch.bfloat16, device="cuda")
        vt = torch.empty_like(kt)
        for i in range(L):
            if i == 0:
                kt[0], vt[0] = self.k0[tok.long()], self.v0[tok.long()]
            else:
                kt[i] = (x @ self.wk[i]).view(B, N, HKV, D).bfloat16()
                vt[i] = (x @ self.wv[i]).view(B, N, HKV, D).bfloat16()
            q = (x @ self.wq[i]).view(B, N, H, D).bfloat16()
            args = (q, s["k"][i], s["v"][i], s["table"], s["lens"], kt[i], vt[i], par, n_nodes)
            o = binding.tree_attention(*args)
            if attend is not None:
                attend(i, args, o)
            x = x + o.float().reshape(B, N, H * D) @ self.wo[i]
        return torch.softmax(x @ self.head, -1), kt, vt


def state(B):
    z = lambda: torch.full((L, PAGES, PS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    return dict(k=z(), v=z(), table=torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda"),
                lens=torch.zeros((B,), dtype=torch.int32, device="cuda"))


def check_attention(i, args, o):
    q, k, v, table, lens, kt, vt, par, nn = args
    h = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    # slots nothing was written to are NaN; the float64 form does not look at them
    want, spread, reach = ref.tree_attention(f64(q), f64(k), f64(v), h(table), h(lens), f64(kt), f64(vt), h(par), h(nn))
    assert np.isfinite(want).all()
    vmax = max(float(np.nanmax(np.abs(f64(v)), initial=0.0)), float(np.abs(f64(vt)).max()))
    tol = attention_tolerance(spread, reach, want, q.dtype, D, vmax)
    assert (np.abs(f64(o) - want) <= tol).all(), i


def check_cache(s, m, history):
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    live = []
    for b, toks in enumerate(history):
        assert lens[b] == len(toks)
        at = np.arange(len(toks))
        live += table[b, :-(-len(toks) // PS)].tolist()
        pages = torch.from_numpy(table[b, at // PS].astype(np.int64)).cuda()
        slots = torch.from_numpy(at % PS).cuda()
        ids = torch.tensor(toks, dtype=torch.int64, device="cuda")
        assert torch.equal(s["k"][0][pages, slots], m.k0[ids]) and torch.equal(s["v"][0][pages, slots], m.v0[ids])
    return live


@pytest.mark.parametrize("drawn", [True, False])
def test_trees_over_several_rounds(drawn):
    B, N, rounds = 6, 9, 6
    m, s = Model(1), state(B)
    rng = np.random.default_rng(2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    root = torch.from_numpy(rng.integers(0, V, B).astype(np.int32)).cuda()
    history = [[] for _ in range(B)]
    said = 0
    for r in range(rounds):
        par_h = parents("random", B, N, rng)
        n_h = rng.integers(1, N + 1, B).astype(np.int32)
        par, nn = dev(par_h), dev(n_h)
        tok = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        tok[:, 0] = root
        q = torch.zeros((B, N, V), device="cuda")
        rows = torch.arange(B, device="cuda")
        order = np.zeros((B, N), np.int64)  # which of its parent's children a node is
        for b in range(B):
            for i in range(1, N):
                order[b, i] = (par_h[b, 1:i] == par_h[b, i]).sum()
        for i in range(N):
            if i:
                up = q[rows, par[:, i].long()]
                if drawn:
                    tok[:, i] = torch.multinomial(up, 1, generator=gen)[:, 0].int()
                else:
                    best = up.topk(N, -1).indices
                    tok[:, i] = best[rows, torch.from_numpy(order[:, i]).cuda()].int()
            q[:, i] = m.draft(tok[:, i])
        p, kt, vt = m.forward(s, tok, par, nn, check_attention)
        ua = torch.from_numpy(rng.random((B, N), np.float32)).cuda()
        uf = torch.from_numpy(rng.random(B, np.float32)).cuda()
        qq = q if drawn else None
        got = binding.verify_tree(p, qq, tok, par, ua, uf, nn)
        h = lambda t: t.cpu().numpy()  # noqa: E731
        t, nd, n, margin = ref.verify_tree(f64(p), None if qq is None else f64(qq), h(tok), par_h, h(ua), h(uf), n_h)
        assert (margin > 1e-8).all()  # sums of 997 float64 terms: rounding below 1e-12
        for a, w in zip(got, (t, nd, n)):
            np.testing.assert_array_equal(h(a), w)
        assert (n >= 0).all()
        s["table"], s["lens"], status = binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], kt, vt, got[1],
                                                             got[2])
        assert int(status) == 0
        for b in range(B):
            history[b] += h(tok)[b, nd[b, :n[b] + 1]].tolist()
        said += int(n.sum())
        root = got[0][torch.arange(B, device="cuda"), got[2].long()]
        live = check_cache(s, m, history)
        assert len(set(live)) == len(live)
    say(f"[tree round] {rounds} rounds, {said} drafted nodes accepted, lengths {[len(x) for x in history]}")
    assert said > 0


def test_chains_with_the_fused_verify():
    """A chain's K + 1 nodes: spec_verify accepts on logits, its counts commit
    the nodes without a node list (an invalid row appends nothing)."""
    B, K = 5, 4
    m, s = Model(5), state(B)
    history = [[] for _ in range(B)]
    par = dev(np.tile(np.arange(-1, K, dtype=np.int32), (B, 1)))
    root = torch.arange(B, dtype=torch.int32, device="cuda") * 31
    gen = torch.Generator(device="cuda").manual_seed(6)
    for r in range(5):
        tok = torch.zeros((B, K + 1), dtype=torch.int32, device="cuda")
        tok[:, 0] = root
        q = torch.zeros((B, K, V), device="cuda")
        for i in range(K):
            q[:, i] = m.draft(tok[:, i])
            tok[:, i + 1] = torch.multinomial(q[:, i], 1, generator=gen)[:, 0].int()
        p, kt, vt = m.forward(s, tok, par, None, check_attention)
        drafted = tok[:, 1:].contiguous()
        if r == 2:
            drafted[1, 0] = V  # not a token: row 1 is invalid in this round
        out, n = binding.verify(torch.log(p), torch.log(q), drafted, None, 1.0, 1.0, 100 + r)
        binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], kt, vt, None, n, out_table=s["table"],
                             out_len=s["lens"])
        nh = n.cpu().numpy()
        assert (nh[1] == -1) == (r == 2)
        for b in range(B):
            history[b] += tok[b, :nh[b] + 1].tolist()
        check_cache(s, m, history)
        ok = n >= 0
        root = torch.where(ok, out[torch.arange(B, device="cuda"), n.clamp(min=0).long()], root)


def test_particles_fork_and_go_on():
    """spec_smc_step's ancestors fork the cache; the particles that share pages
    then grow apart, and dropped particles' pages are used again."""
    B, K = 8, 3
    m, s = Model(7), state(B)
    history = [[] for _ in range(B)]
    par = dev(np.tile(np.arange(-1, K, dtype=np.int32), (B, 1)))
    all_nodes = torch.full((B,), K, dtype=torch.int32, device="cuda")
    root = torch.full((B,), 11, dtype=torch.int32, device="cuda")
    logw = torch.zeros((B,), dtype=torch.float64, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(8)
    moved = 0
    for r in range(8):
        tok = torch.zeros((B, K + 1), dtype=torch.int32, device="cuda")
        tok[:, 0] = root
        q = torch.zeros((B, K, V), device="cuda")
        for i in range(K):
            q[:, i] = m.draft(tok[:, i])
            tok[:, i + 1] = torch.multinomial(q[:, i], 1, generator=gen)[:, 0].int()
        p, kt, vt = m.forward(s, tok, par, None, check_attention)
        s["table"], s["lens"], status = binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], kt, vt, None,
                                                             all_nodes)
        assert int(status) == 0
        for b in range(B):
            history[b] += tok[b].tolist()
        bonus, logw, anc, _, resampled = binding.smc_step(torch.log(p), torch.log(q), tok[:, 1:].contiguous(), logw, 1.0,
                                                          0.9, 50 + r)
        k, v = s["k"].clone(), s["v"].clone()
        want = ref.cache_fork(*[t.view(torch.int16).cpu().numpy() for t in (k, v)], s["table"].cpu().numpy(),
                              s["lens"].cpu().numpy(), anc.cpu().numpy())
        s["table"], s["lens"], status = binding.cache_fork(s["k"], s["v"], s["table"], s["lens"], anc)
        assert int(status) == want[2] == 0
        np.testing.assert_array_equal(s["table"].cpu().numpy(), want[0])
        a = anc.tolist()
        moved += sum(x != b for b, x in enumerate(a))
        history = [list(history[x]) for x in a]
        root = bonus[anc.long()]
        check_cache(s, m, history)
        assert (s["lens"] <= WIDTH * PS).all()
    say(f"[tree round] particles: {moved} slots took another's sequence")
    assert moved > 0


def test_whole_round_captured():
    """Attention, verification and an in-place commit in one graph, replayed
    while the lengths grow, against eager rounds on a copy of the state."""
    B, N = 4, 7
    m = Model(9)
    eager, fixed = state(B), state(B)
    par = dev(parents("level2", B, N, np.random.default_rng(0)))
    keep = {k: v.clone() for k, v in fixed.items()}
    stream = torch.cuda.Stream()

    def one(s, tok, ua, uf):
        p, kt, vt = m.forward(s, tok, par)
        out = binding.verify_tree(p, None, tok, par, ua, uf)
        return (*out, *binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], kt, vt, out[1], out[2],
                                            out_table=s["table"], out_len=s["lens"]))

    rng = np.random.default_rng(4)
    new = lambda: (dev(rng.integers(0, V, (B, N)).astype(np.int32)), dev(rng.random((B, N), np.float32)),  # noqa: E731
                   dev(rng.random(B, np.float32)))
    bufs = new()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        one(fixed, *bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = one(fixed, *bufs)
    torch.cuda.synchronize()
    for k, v in keep.items():
        fixed[k].copy_(v)
    for rep in range(6):
        inputs = new()
        for b, x in zip(bufs, inputs):
            b.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = one(eager, *inputs)
        torch.cuda.synchronize()
        for g, w in zip(outs, want):
            assert torch.equal(g, w), rep
        for name in ("k", "v"):
            assert torch.equal(fixed[name].view(torch.int16), eager[name].view(torch.int16)), rep
    assert (fixed["lens"] >= 6).all()


def test_a_count_past_the_tree_appends_nothing():
    B, N = 3, 4
    s = state(B)
    kt = torch.zeros((L, B, N, HKV, D), dtype=torch.bfloat16, device="cuda")
    for n in (N, 2 ** 31 - 1):
        counts = torch.tensor([0, n, 1], dtype=torch.int32, device="cuda")
        table, lens, status = binding.cache_commit(s["k"], s["v"], s["table"], s["lens"], kt, kt, None, counts)
        assert int(status) == -1 and int(lens.abs().sum()) == 0 and bool((table == -1).all())
        assert bool(torch.isnan(s["k"]).all())


def test_first_call_of_a_process_captured():
    """Nothing has to run before the first capture."""
    code = '''
import torch
from rejection_sampling_verifier_amd import binding as b
z = lambda *s: torch.randn(s, device="cuda").bfloat16()
i = lambda v, *s: torch.full(s, v, dtype=torch.int32, device="cuda")
q, kc, vc, kt, vt = z(2, 3, 8, 128), z(1, 40, 64, 2, 128), z(1, 40, 64, 2, 128), z(1, 2, 3, 2, 128), z(1, 2, 3, 2, 128)
table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
lens, par = i(700, 2), i(0, 2, 3)
p, u = torch.softmax(torch.randn((2, 3, 30000), device="cuda"), -1), torch.rand((2, 3), device="cuda")
tok, uf = i(7, 2, 3), u[:, 0].contiguous()
torch.cuda.synchronize()
def step():
    o = b.tree_attention(q, kc[0], vc[0], table, lens, kt[0], vt[0], par)
    t = b.verify_tree(p, p[:, :1], tok, par, u, uf)
    c = b.cache_commit(kc, vc, table, lens, kt, vt, t[1], t[2])
    f = b.cache_fork(kc, vc, c[0], c[1], par[:, 0].contiguous())
    return (o, *t, *c, *f)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = step()
for _ in range(3):
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, step()):
        assert torch.equal(x, y)
torch.cuda.synchronize()
print("captured")
'''
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured" in r.stdout, (r.returncode, r.stderr[-2000:])
