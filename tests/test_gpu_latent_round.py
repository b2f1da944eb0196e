"""Beam decoding with a latent-attention model, call by call as a decoder runs
it: pages for the prompts, their rows written, the prompts' attention, the first
selection with the pages forked; then steps of one token per beam (products into
the latent space, attention on the rows, products out of it, selection, fork,
histories reordered).  Every call is compared with the oracle on the inputs it
had, the cache must hold the histories' rows, and a captured step replays as the
eager one."""

import numpy as np
import pytest
import torch

import test_gpu_beam as bm
import test_gpu_latent_attention as att
import test_gpu_latent_prompt as pro
import test_gpu_reserve as rsv
from oracle import latent as ref
from oracle import tree as ref_tree
from rejection_sampling_verifier_amd import binding
from tree_helpers import f64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
B, W, V = 3, 4, 1000
H, DN, DR, DV, R, PS = 5, 32, 16, 40, 112, 8
C, PAGES, WIDTH, END = R + DR, 90, 12, 7
SCALE = (DN + DR) ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


class Model:
    """One layer: a token's query and row come from tables, the row's second part
    turned by its position; logits are the attention's output times a matrix."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(0)
        r = lambda *s, by=1.0: (torch.randn(s, generator=g, device="cuda") * by).to(BF16)  # noqa: E731
        self.q, self.row = r(V, H, DN + DR, by=2.0), r(V, C)
        self.w_k, self.w_v = r(H, DN, R, by=R ** -0.5), r(H, DV, R, by=R ** -0.5)
        self.w_in = self.w_k.transpose(1, 2).contiguous()  # laid out once: queries into the latent space
        self.head = r(1, V, H * DV, by=0.5)

    def rows(self, tokens, position):
        """(latent part, positions' part) of tokens at positions."""
        x = self.row[tokens.long()]
        turn = torch.cos(position.float()[:, None] * torch.arange(1, DR + 1, device="cuda") * 0.1)
        return x[:, :R].contiguous(), (x[:, R:].float() * turn).to(BF16)


def halves(cache):
    """The cache as cache_fork takes it: one layer, one head, the row's two halves."""
    c = cache[None, :, :, None]
    return c[..., :C // 2], c[..., C // 2:]


def checked_fork(cache, table, lens, anc):
    k, v = halves(cache)
    before = [t.cpu().numpy() for t in (table, lens, anc)]
    want_k, want_v = (t.float().cpu().numpy() for t in (k, v))
    out = binding.cache_fork(k, v, table, lens, anc)
    torch.cuda.synchronize()
    want = ref_tree.cache_fork(want_k, want_v, *before[:2], before[2])
    for a, b in zip(out, want):
        np.testing.assert_array_equal(a.cpu().numpy(), np.atleast_1d(b))
    for a, b in zip((k, v), (want_k, want_v)):
        np.testing.assert_array_equal(a.float().cpu().numpy(), b)
    assert int(out[2]) == 0
    return out[0], out[1]


def step(m, cache, table, lens, tokens, scores, done, history, check=False):
    """One token per beam; returns the state after it."""
    n = B * W
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    flat = tokens.view(-1).clamp(0)
    q = m.q[flat.long()]
    latent, turned = m.rows(flat, lens)
    new = torch.cat((latent, turned), 1)[:, None]
    product = pro.product_check if check else lambda x, w, label: binding.head_product(x, w)
    into = product(q[..., :DN], m.w_in, "into the latent space")
    q = torch.cat((into, q[..., DN:]), -1)[:, None]
    s = dict(q=q, cache=cache, rows=new, table=table, lens=lens, parent=None, n_nodes=None, dv=R, scale=SCALE)
    mid = att.check(s, "decoding") if check else att.call(s)
    if check:
        rsv.check(table.cpu().numpy(), lens.cpu().numpy(), ones.cpu().numpy(), PAGES, PS, n)
    table, lens, _, slots, _, status = binding.cache_reserve(table, lens, ones, pages=PAGES, page_size=PS, rows=n)
    binding.cache_write(cache, slots, latent, turned)
    out = product(mid[:, 0], m.w_v, "out of the latent space")
    logits = product(out.view(n, 1, H * DV), m.head, "logits").view(B, W, V)
    pick = bm.check if check else lambda *a, end, label: binding.beam_select(*a, end=end)
    tokens, anc, scores, done = pick(logits, scores, done, end=END, label="selection")
    if check:
        table, lens = checked_fork(cache, table, lens, anc)
    else:
        table, lens, _ = binding.cache_fork(*halves(cache), table, lens, anc)
    history = binding.beam_reorder(history, anc)
    return table, lens, tokens, scores, done, history, status


def prefill(m, check=False):
    """Three prompts in the first beam's place of each sequence."""
    g = torch.Generator(device="cuda").manual_seed(4)
    counts = np.zeros(B * W, np.int32)
    counts[::W] = (19, 1, 33)
    T = int(counts.sum())
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    cache = torch.full((PAGES, PS, C), float("nan"), dtype=BF16, device="cuda")
    table = torch.full((B * W, WIDTH), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    if check:
        rsv.check(table.cpu().numpy(), lens.cpu().numpy(), counts, PAGES, PS, T)
    table, lens, start, slots, position, status = binding.cache_reserve(
        table, lens, torch.from_numpy(counts).cuda(), pages=PAGES, page_size=PS, rows=T)
    assert int(status) == 0
    binding.cache_write(cache, slots, *m.rows(tokens, position))
    s = dict(q=m.q[tokens.long()], cache=cache, table=table, lens=lens, start=start, w_k=m.w_k, w_v=m.w_v, rows=T)
    out = pro.check(s, "prompts") if check else pro.call(s)
    logits = torch.zeros((B, W, V), dtype=BF16, device="cuda")
    last = start.long()[1:][::W] - 1
    logits[:, 0] = binding.head_product(out[last].reshape(B, 1, H * DV), m.head)[:, 0]
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros((B, W), dtype=torch.int32, device="cuda")
    picked = bm.check(logits, scores, done, end=END, label="first") if check else \
        binding.beam_select(logits, scores, done, end=END)
    table, lens = checked_fork(cache, table, lens, picked[1])
    prompts = [tokens[start[W * b]:start[W * b] + counts[W * b]].tolist() for b in range(B)]
    history = picked[0].view(-1, 1).expand(-1, 16).contiguous()
    return cache, table, lens, *((picked[0],) + picked[2:]), history, prompts


def test_decoding():
    m = Model()
    cache, table, lens, tokens, scores, done, history, prompts = prefill(m, check=True)
    for i in range(5):
        history[:, i] = tokens.view(-1)
        table, lens, tokens, scores, done, history, status = step(m, cache, table, lens, tokens, scores, done, history,
                                                                  check=True)
        assert int(status) == 0 and (scores[:, :-1] >= scores[:, 1:]).all()
        # the cache holds, for every beam, its prompt's rows and those of the tokens it went through
        for k in range(B * W):
            path = prompts[k // W] + history[k, :i + 1].tolist()
            n = int(lens[k])
            assert n == len(path)
            j = torch.arange(n, device="cuda")
            want = torch.cat(m.rows(torch.tensor(path, device="cuda").clamp(0), j), 1)
            assert torch.equal(cache[table[k, j // PS].long(), j % PS], want), (i, k)
    assert len(set(map(tuple, history[:, :5].tolist()))) > B


def test_expanded_and_absorbed_agree():
    """The newest token of every beam through either form, each against float64.
    With h half a step of the type: a key's rounding (expanded) or the absorbed
    query's moves a score by at most h times the sum of its terms' sizes, and a
    weight by twice that; weights and values are rounded once, the result in the
    latent space (absorbed) and the output once.  A twentieth on top is above all
    second orders and float32 sums of these few rows."""
    m = Model()
    cache, table, lens, tokens, *_ = prefill(m)
    n, h = B * W, 2.0 ** -8
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    q = m.q[tokens.view(-1).clamp(0).long()]
    expanded = f64(binding.latent_prompt(q, cache, table, lens, start, m.w_k, m.w_v, rows=int(lens.sum())))
    # the last row is the node's own; before it the cache
    j = lens.long() - 1
    own = cache[table.gather(1, (j // PS)[:, None])[:, 0].long(), j % PS][:, None]
    into = binding.head_product(q[..., :DN], m.w_in)
    mid = binding.latent_attention(torch.cat((into, q[..., DN:]), -1)[:, None], cache, table, lens - 1, own, dim_v=R,
                                   scale=SCALE)[:, 0]
    absorbed = f64(binding.head_product(mid, m.w_v))
    host = [t.cpu().numpy() for t in (table, lens, start)]
    want, spread, reach, _ = ref.prompt(f64(q), f64(cache), *host, f64(m.w_k), f64(m.w_v), SCALE)
    size = np.zeros((n, H, 1))
    for k in range(n):
        rows = np.abs(ref.cache_rows(f64(cache), host[0][k], host[1][k]))[:, :R]
        size[k, :, 0] = SCALE * (np.abs(f64(into))[k] @ rows.T).max(-1)
    sums = ref.head_product(np.abs(f64(mid)), np.abs(f64(m.w_v)))[0]
    tol = 1.05 * h * (2 * spread + np.abs(want)) + np.expm1(2.1 * h * reach[..., :1]) * spread
    assert (np.abs(expanded - want) <= tol).all()
    tol = 1.05 * h * (spread + sums + np.abs(want)) + np.expm1(2.1 * h * size) * spread
    assert (np.abs(absorbed - want) <= tol).all()


def test_captured_steps():
    """A captured step, state to state in place, against the eager one: four replays
    with eager work between them."""
    m = Model()
    cache, *state, _ = prefill(m)
    state = [t.clone() for t in state]
    state[1:] = [t.contiguous() for t in state[1:]]
    for t in step(m, cache.clone(), *state):  # once, so that nothing is set up while capturing
        assert t is not None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    kept = cache.clone()
    with torch.cuda.graph(graph):
        after = step(m, kept, *state)
        for a, b in zip(state, after):
            a.copy_(b)
    eager, mine = cache.clone(), [t.clone() for t in state]
    for rep in range(4):
        mine = list(step(m, eager, *mine)[:6])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(state, mine):
            assert torch.equal(a, b), rep
        live = eager.isfinite()
        assert torch.equal(live, kept.isfinite()) and torch.equal(eager[live], kept[live]), rep
