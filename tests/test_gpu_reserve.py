"""spec_cache_reserve and spec_cache_write on the GPU against the oracle, exact
in every byte: new requests, single rows, shared and full pages, refusals on the
device, large pools and batches, in-place tables, strides."""

import numpy as np
import pytest
import torch

from oracle import beam as ref
from rejection_sampling_verifier_amd import binding
from tree_helpers import dev, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


def check(table, lens, new, pages, ps, rows, **kw):
    want = ref.cache_reserve(table, lens, np.asarray(new), pages, ps, rows)
    t, n = kw.pop("t", None), kw.pop("n", None)
    t, n = dev(table) if t is None else t, dev(np.asarray(lens, np.int32)) if n is None else n
    got = binding.cache_reserve(t, n, dev(np.asarray(new, np.int32)), pages=pages, page_size=ps, rows=rows, **kw)
    torch.cuda.synchronize()
    for name, a, b in zip(("table", "len", "start", "slots", "position", "status"), got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), np.atleast_1d(b), err_msg=name)
    return got


def make(lens, new, ps, spare, seed=0):
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    pages, table = tables(lens, ps, rng, extra=int(new.max(initial=0)) // ps + 1, spare=spare)
    return table, lens, new, pages, ps, int(np.maximum(new, 0).sum()) + 5


@pytest.mark.parametrize("ps", [1, 2, 16, 64, 1024])
@pytest.mark.parametrize("B", [1, 7, 64, 300])
def test_batches(ps, B):
    rng = np.random.default_rng(B + ps)
    lens, new = rng.integers(0, 300, B), rng.integers(0, 200, B)
    check(*make(lens, new, ps, spare=int((new // ps + 2).sum()), seed=ps))


@pytest.mark.parametrize("lens,new", [((0,), (1,)), ((0,), (0,)), ((16,), (1,)), ((15,), (1,)), ((15,), (2,)),
                                      ((0, 0), (4096, 1)), ((31, 32, 33), (0, 0, 0)), ((5, 9), (-3, 40))])
def test_single_rows_and_borders(lens, new):
    check(*make(lens, new, 16, spare=300))


def test_more_sequences_than_threads():
    rng = np.random.default_rng(8)
    lens, new = rng.integers(0, 40, 2500), rng.integers(0, 3, 2500)
    lens[1700] = 5000
    check(*make(lens, new, 8, spare=3000))


@pytest.mark.parametrize("pages", [1000, 1024, 1025, 2048, 70000, 1 << 20])
def test_pool_sizes(pages):
    """Free pages at both ends of the pool and in between."""
    rng = np.random.default_rng(pages)
    used = rng.permutation(pages)[:min(pages - 300, 5000)].astype(np.int32)
    table = np.full((5, 1400), -1, np.int32)
    table.reshape(5, -1)[:, :len(used) // 5] = used[:len(used) // 5 * 5].reshape(5, -1)
    lens = np.full(5, len(used) // 5 * 4, np.int32)
    check(table, lens, [33, 1, 0, 700, 2], pages, 4, 800)


def test_whole_pool_and_one_page_too_few():
    # 2 + 1 pages are used and 4 free; 2 more and 1 more are needed, then 2 and 2, then 2 and 3
    table, lens, new, pages, ps, rows = make((30, 7), (34, 25), 16, spare=4)
    check(table, lens, new, pages, ps, rows)
    table = np.concatenate([table, np.full((2, 20), -1, np.int32)], 1)
    assert int(check(table, lens, [34, 41], pages, ps, 400)[5]) == 0
    assert int(check(table, lens, [34, 42], pages, ps, 400)[5]) == 1
    assert int(check(table, lens, [34, 25 + 16 * 9], pages, ps, 400)[5]) > 1


def test_table_row_too_short():
    table, lens, new, pages, ps, rows = make((30, 7), (34, 25), 16, spare=4)
    assert int(check(table, lens, [34, 25 + 16 * 9], pages, ps, 400)[5]) == -1


def test_shared_pages():
    """Full pages may be shared; a partly filled one that is appended to may not."""
    table = np.array([[3, 5, -1, -1], [3, 6, -1, -1], [3, 5, -1, -1]], np.int32)
    check(table, np.array([20, 30, 16], np.int32), [4, 4, 4], 10, 16, 20)  # row 2's second entry is not live
    got = check(table, np.array([20, 30, 20], np.int32), [0, 4, 4], 10, 16, 20)
    assert int(got[5]) == -1
    check(table, np.array([20, 30, 20], np.int32), [0, 4, 0], 10, 16, 20)


@pytest.mark.parametrize("lens,new,rows", [((-1, 5), (1, 1), 9), ((65, 5), (0, 1), 9), ((60, 5), (5, 1), 9),
                                           ((5, 5), (4, 6), 9), ((5, 5), (2 ** 31 - 1, 2 ** 31 - 1), 9)])
def test_out_of_range(lens, new, rows):
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7]], np.int32)
    got = check(table, np.array(lens, np.int32), new, 40, 16, rows)
    assert int(got[5]) == -1


@pytest.mark.parametrize("page", [-1, 40, 2 ** 31 - 1])
def test_bad_live_page(page):
    table = np.array([[0, page, 2, 3], [4, 5, 6, 7]], np.int32)
    assert int(check(table, np.array([30, 9], np.int32), [1, 1], 40, 16, 9)[5]) == -1
    check(table, np.array([16, 9], np.int32), [1, 1], 40, 16, 9)  # not live: not looked at


def test_in_place_and_strided():
    table, lens, new, pages, ps, rows = make((30, 0, 200), (3, 100, 60), 16, spare=40)
    wide = torch.full((3, table.shape[1] + 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = dev(table)
    t, n = wide[:, 2:2 + table.shape[1]], dev(lens)
    got = check(table, lens, new, pages, ps, rows, t=t, n=n, out_table=t, out_len=n)
    assert got[0] is t and got[1] is n and (wide[:, :2] == 77).all() and (wide[:, 2 + table.shape[1]:] == 77).all()


def test_no_rows():
    t, n, start, slots, position, status = check(*make((17, 3), (0, 0), 16, spare=1)[:5], 0)
    assert slots.shape == (0,) and int(status) == 0


# ---- rows into their slots

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T", [1, 5, 700])
@pytest.mark.parametrize("da,db", [(512, 64), (8, 0), (24, 8)])
def test_write(dtype, T, da, db):
    g = torch.Generator(device="cuda").manual_seed(T)
    pages, ps = T // 8 + 3, 16
    cache = torch.randn((pages, ps, da + db), generator=g, device="cuda").to(dtype)
    a, b = (torch.randn((T, d), generator=g, device="cuda").to(dtype) for d in (da, db))
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::4] = -1
    slots[2::8] = pages * ps
    want = cache.clone().view(pages * ps, -1)
    keep = (slots >= 0) & (slots < pages * ps)
    want[slots[keep].long()] = torch.cat((a, b), 1)[keep]
    assert binding.cache_write(cache, slots, a, b if db else None) is None
    assert torch.equal(cache.view(pages * ps, -1), want)


def test_write_strided():
    """A layer of a cache, slots before pages, slices of wider activations."""
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn((16, 5, 2, 40), generator=g, device="cuda").to(torch.bfloat16)
    cache = pool[:, :, 1].transpose(0, 1)[:, :, 8:]  # [5 pages, 16 slots, 32]
    x = torch.randn((11, 72), generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(80, generator=g, device="cuda")[:11].to(torch.int32)
    want = pool.clone()
    for t, s in enumerate(slots.tolist()):
        want[s % 16, s // 16, 1, 8:] = torch.cat((x[t, 16:40], x[t, 64:72]))
    binding.cache_write(cache, slots, x[:, 16:40], x[:, 64:72])
    assert torch.equal(pool, want)


def test_write_nothing():
    cache = torch.zeros((2, 4, 16), dtype=torch.float16, device="cuda")
    binding.cache_write(cache, torch.zeros(0, dtype=torch.int32, device="cuda"), cache.new_empty((0, 16)))
    assert (cache == 0).all()
