"""Request layout on the GPU against a loop over requests (exact)."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def make(rng, B, page, max_blocks, n_free, begin, T, long=False):
    cached = rng.integers(0, max_blocks * page, B)
    cached[rng.random(B) < 0.2] = 0
    new = np.where(rng.random(B) < 0.3, 0, 1)
    if long:
        for b in rng.integers(0, B, max(1, B // 20)):
            new[b] = rng.integers(1, max_blocks * page)
    cached = np.minimum(cached, max_blocks * page - new)
    n_pages = B * max_blocks + n_free + 3
    perm = rng.permutation(n_pages).astype(np.int32)
    table = perm[:B * max_blocks].reshape(B, max_blocks).copy()
    return cached.astype(np.int32), new.astype(np.int32), table, perm[B * max_blocks:][:n_free].copy(), begin, n_pages, page, T


def run(x, status=True):
    cached, new, table, free, begin, n_pages, page, T = x
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    tab = g(table)
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
    r = dsa.dsa_block_tables(g(cached), g(new), tab, g(free), torch.tensor([begin], dtype=torch.int32, device="cuda"),
                             n_pages, page, T, status=st)
    torch.cuda.synchronize()
    return [a.cpu().numpy() for a in r] + [tab.cpu().numpy(), int(st) if status else 0]


def check(x):
    got, want = run(x), ref.block_tables(x[0], x[1], x[2], x[3], x[4], *x[5:])
    for name, g, w in zip(("slot", "position", "owner", "row_start", "seq_len"), got, want):
        assert np.array_equal(g, w), name
    assert int(got[5][0]) == want[5] and np.array_equal(got[6], want[6])
    assert got[7] == (2 if want[7] else 0)


@pytest.mark.parametrize("B,page,max_blocks,long", [
    (1, 64, 4, False), (1, 1, 7, True), (3, 16, 5, True), (31, 64, 9, True), (64, 64, 33, False), (255, 192, 4, True),
    (256, 64, 3, True), (257, 64, 3, True), (1000, 100, 3, True), (1025, 64, 2, False), (5000, 48, 2, True),
])
def test_layout(B, page, max_blocks, long):
    rng = np.random.default_rng(B * 1000 + page)
    x = make(rng, B, page, max_blocks, B * max_blocks + 5, 3, 0, long)
    total = int(x[1].sum())
    for T in {total, total + 1, total + 777}:
        check(x[:7] + (T,))


def test_layout_edges():
    rng = np.random.default_rng(7)
    x = list(make(rng, 40, 64, 4, 200, 2, 100))
    x[1][:] = 0                                     # nothing new at all
    check(x)
    check(x[:7] + [0])                              # and no row
    x[0][:], x[1][:] = 0, 64 * 4                    # every request fills its table
    x[3] = np.arange(170, dtype=np.int32)
    check(x[:7] + [40 * 256])
    x[4] = 10                                       # the free list ends exactly
    check(x[:7] + [40 * 256])


def test_layout_all_or_nothing():
    rng = np.random.default_rng(8)
    base = make(rng, 300, 64, 4, 1300, 0, 2000, False)
    for change in ("rows", "pages", "long", "negative", "negative_new", "begin", "begin_past", "huge"):
        x = [a.copy() if isinstance(a, np.ndarray) else a for a in base]
        if change == "rows":
            x[7] = int(x[1].sum()) - 1
        elif change == "pages":
            x[0][:], x[1][:] = 0, 65
            x[7], x[3] = 300 * 65, x[3][:599]       # one page short
        elif change == "long":
            x[0][211], x[1][211] = 64 * 4, 1
        elif change == "negative":
            x[0][5] = -1
        elif change == "negative_new":
            x[1][299] = -3
        elif change == "begin":
            x[4] = -1
        elif change == "begin_past":
            x[4] = len(x[3]) + 1
        elif change == "huge":
            x[0][:] = x[1][:] = 2 ** 31 - 1         # sums past 32 bits
        want = ref.block_tables(*x)
        if change != "begin_past" or want[7]:
            assert want[7], change
        check(x)


def test_layout_flags_bad_pages_and_leaves_other_entries():
    rng = np.random.default_rng(9)
    x = list(make(rng, 20, 64, 4, 100, 0, 64))
    x[0][:], x[1][:] = 65, 1
    x[2][3, 1] = -1                                 # the partly filled block has no page
    x[2][4, 1] = x[5]                               # and one past the pool
    x[0][7], x[1][7] = 64, 1
    x[3][0] = x[5] + 9                              # a free page that does not exist
    check(x)
    got = run(x, status=False)                      # without a status word: the same
    assert got[0][3] == got[0][4] == got[0][7] == -1


def test_layout_replays_in_a_graph():
    rng = np.random.default_rng(10)
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    a, b = (make(np.random.default_rng(s), 50, 64, 6, 400, 1, 90) for s in (11, 12))
    n_pages = max(a[5], b[5])
    cached, new, tab, free = (g(v) for v in a[:4])
    begin = torch.tensor([1], dtype=torch.int32, device="cuda")
    outs = dsa.dsa_block_tables(cached, new, tab, free, begin, n_pages, 64, 90)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_block_tables(cached, new, tab, free, begin, n_pages, 64, 90, *outs)
    for x in (b, a):
        for dst, src in zip((cached, new, tab, free), x[:4]):
            dst.copy_(g(src))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.block_tables(*x[:5], n_pages, 64, 90)
        for got, w in zip(outs, want[:5]):
            assert np.array_equal(got.cpu().numpy(), w)
        assert np.array_equal(tab.cpu().numpy(), want[6])


@pytest.mark.parametrize("B,page,max_blocks", [(2049, 7, 3), (4095, 64, 2), (4096, 1, 5), (4097, 64, 2)])
def test_layout_many_requests(B, page, max_blocks):
    # up to and past the number of requests whose sums one block keeps
    test_layout(B, page, max_blocks, True)
