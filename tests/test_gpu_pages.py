"""mq_pages_next and mq_pages_compact against plain forms on lists: tables, lengths, status and every byte of the pool."""
import random

import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests import _kv4_ref as R
from tests._gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dev(x):
    return None if x is None else torch.tensor(x, dtype=I32, device="cuda")


def _pool(layers, P, size, rows, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    raw = torch.randint(0, 256, (layers, P, size), generator=g, device="cuda", dtype=torch.uint8)
    return raw, mq.Pool(raw, rows)


def _tables(n, width, rows, P, r, shared=0.3, holes=0.0):
    """Sequences that share some of their first pages, as forks leave them."""
    free = list(range(P))
    r.shuffle(free)
    table, length = [], []
    for b in range(n):
        L = r.randint(0, width * rows)
        used = -(-L // rows)
        row = [-1] * width
        src = table[r.randrange(b)] if b and r.random() < shared else None
        for j in range(used):
            if src and src[j] >= 0 and j < max(1, used - 1):
                row[j] = src[j]
            elif free:
                row[j] = free.pop()
            if r.random() < holes:
                row[j] = r.choice([-1, P, P + 7, -2 ** 31, 2 ** 31 - 1])
        table.append(row)
        length.append(L)
    return table, length


def _next(table, length, m, P, rows, frm=None, keep=None, add=None, layers=2, size=160, in_place=False, seed=0):
    raw, pool = _pool(layers, P, size, rows, seed)
    width = len(table[0])
    want = R.next_pages(table, length, frm, keep, add, P, rows, m)
    old = raw.clone()
    t, n = _dev(table), _dev(length)
    t_out, n_out = Guarded((m, width), I32), Guarded((m,), I32)
    status = Guarded((3,), I32)
    if in_place:
        mq.mq_pages_next(pool, t, n, t, n, status.t, _dev(frm), _dev(keep), _dev(add))
        got_t, got_n = t, n
    else:
        mq.mq_pages_next(pool, t, n, t_out.t, n_out.t, status.t, _dev(frm), _dev(keep), _dev(add))
        got_t, got_n = t_out.t, n_out.t
        assert t.tolist() == table and n.tolist() == length
        t_out.check()
        n_out.check()
    torch.cuda.synchronize()
    status.check()
    assert status.t.tolist() == want[2]
    assert got_n.tolist() == want[1]
    assert got_t.tolist() == want[0]
    for a, b in want[3]:
        old[:, b] = old[:, a]
    assert torch.equal(raw, old)
    return want


@pytest.mark.parametrize("n,width,rows,P", [(1, 1, 16, 1), (1, 7, 16, 9), (5, 4, 32, 30), (70, 9, 64, 700), (300, 40, 16, 9000),
                                            (3, 1000, 16, 4000), (9000, 3, 16, 40000)])
@pytest.mark.parametrize("kind", ["reserve", "fork", "trim", "all", "in place"])
def test_next(n, width, rows, P, kind):
    r = random.Random(n + len(kind))
    table, length = _tables(n, width, rows, P, r, shared=0.0 if kind in ("reserve", "in place") else 0.3)
    m = n if kind in ("reserve", "trim", "in place") else max(1, n + r.randint(-3, 5))
    frm = None if kind in ("reserve", "in place") else [r.randint(-1, n) for _ in range(m)]
    keep = None if kind in ("reserve", "fork") else [r.randint(-2, width * rows) for _ in range(m)]
    add = None if kind == "trim" else [r.choice([0, 1, 1, 2, rows, r.randint(0, 2 * rows), -3]) for _ in range(m)]
    _next(table, length, m, P, rows, frm, keep, add, in_place=kind == "in place", seed=n)


def test_next_beams():
    """All beams of a prompt go on: the first keeps the page, the others get copies; one that does not go on stays on it."""
    rows, width, P = 16, 4, 24
    table, length = [[3, 9, 2, -1], [5, -1, -1, -1]], [37, 16]
    w = _next(table, length, 5, P, rows, [0, 0, 0, 1, 1], None, [1, 1, 1, 1, 1])
    assert [a for a, _ in w[3]] == [2, 2] and w[0][0][2] == 2
    w = _next(table, length, 3, P, rows, [0, 0, 0], None, [1, 0, 2])
    assert len(w[3]) == 2 and w[0][1][2] == 2
    w = _next(table, length, 2, P, rows, [0, 0], [37, 34], [1, 1])       # trimmed inside the same page
    assert len(w[3]) == 1
    w = _next(table, length, 2, P, rows, [0, 0], [32, 32], [1, 1])       # at a page's end: nothing to copy
    assert w[3] == []


def test_next_too_few_pages():
    table, length = [[0, 1, -1, -1], [2, -1, -1, -1]], [32, 3]
    w = _next(table, length, 2, 4, 16, None, None, [20, 1])             # two wanted, one free
    assert w[2] == [1, 1, 0] and w[1] == [32, 3]
    w = _next(table, length, 2, 4, 16, None, None, [16, 1])
    assert w[2] == [0, 0, 0]
    w = _next(table, length, 2, 4, 16, None, None, [33, 1])             # past the table: none, the others are served
    assert w[2] == [0, 1, 1] and w[1] == [32, 4]
    w = _next(table, length, 3, 4, 16, [1, 1, 1], None, [1, 1, 1])
    assert w[2] == [0, 1, 0]


@pytest.mark.parametrize("seed", range(4))
def test_next_holes(seed):
    r = random.Random(seed)
    table, length = _tables(20, 6, 16, 90, r, holes=0.2)
    _next(table, length, 25, 90, 16, [r.randint(-1, 20) for _ in range(25)], None, [r.randint(0, 20) for _ in range(25)])
    _next(table, [-4, 10 ** 9] + length[2:], 20, 200, 16, None, None, [1] * 20)


@pytest.mark.parametrize("layers,size", [(1, 16), (3, 16368), (2, 16384), (5, 16400), (1, 1 << 20)])
def test_next_page_sizes(layers, size):
    _next([[1, 2, -1]], [20], 3, 9, 16, [0, 0, 0], None, [1, 2, 3], layers=layers, size=size)


def test_pool_strides():
    """Pages of layers, and a slice of a wider pool."""
    P, layers, size = 12, 3, 96
    raw = torch.randint(0, 256, (P, layers, size + 32), device="cuda", dtype=torch.uint8)
    old = raw.clone()
    pool = mq.Pool(raw[:, :, 16:16 + size].transpose(0, 1), 16)
    t, n = _dev([[4, 5]]), _dev([20])
    t_out, n_out, status = torch.zeros((2, 2), dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda"), torch.zeros(3, dtype=I32, device="cuda")
    mq.mq_pages_next(pool, t, n, t_out, n_out, status, _dev([0, 0]), None, _dev([1, 1]))
    assert t_out.tolist() == [[4, 5], [4, 0]]
    old[0, :, 16:16 + size] = old[5, :, 16:16 + size]
    assert torch.equal(raw, old)


@pytest.mark.parametrize("n,width,rows,P", [(1, 1, 16, 1), (1, 3, 16, 50), (7, 5, 32, 60), (40, 30, 16, 3000), (2, 3000, 16, 20000),
                                            (5000, 4, 16, 30000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n, width, rows, P, in_place):
    r = random.Random(n)
    table, length = _tables(n, width, rows, P, r, holes=0.02)
    raw, pool = _pool(2, P, 112, rows, n)
    old = raw.clone()
    out, where, live, moves = R.compact_pages(table, length, P, rows)
    t, n_dev = _dev(table), _dev(length)
    t_out = t if in_place else Guarded((n, width), I32).t
    w, u = Guarded((P,), I32), Guarded((1,), I32)
    mq.mq_pages_compact(pool, t, n_dev, t_out, w.t, u.t)
    torch.cuda.synchronize()
    w.check()
    u.check()
    assert u.t.tolist() == [live] and w.t.tolist() == where and t_out.tolist() == out
    for a, b in moves:
        old[:, b] = old[:, a]
    assert torch.equal(raw, old)


def test_compact_all_or_nothing():
    for table, length, P in (([[0, 1], [2, 3]], [32, 32], 4), ([[0, 1]], [0], 4), ([[3, 3], [3, 0]], [32, 17], 4)):
        raw, pool = _pool(1, P, 32, 16)
        want = R.compact_pages(table, length, P, 16)
        old = raw.clone()
        t, w, u = _dev(table), torch.zeros(P, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
        mq.mq_pages_compact(pool, t, _dev(length), t, w, u)
        assert t.tolist() == want[0] and w.tolist() == want[1] and u.tolist() == [want[2]]
        for a, b in want[3]:
            old[:, b] = old[:, a]
        assert torch.equal(raw, old)


def test_in_a_graph_and_on_a_stream():
    """Reserve, captured, in place: a table that grows replay by replay."""
    rows, width, P, n = 16, 5, 20, 3
    raw, pool = _pool(2, P, 64, rows)
    table, length = [[-1] * width for _ in range(n)], [0] * n
    t, ln, status, add = _dev(table), _dev(length), torch.zeros(3, dtype=I32, device="cuda"), _dev([7, 16, 1])
    ws = mq.pages_workspace(pool, n, width)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mq.mq_pages_next(pool, t, ln, t, ln, status, add=add, ws=ws, stream=side)
    torch.cuda.synchronize()
    table, length, st, _ = R.next_pages(table, length, None, None, [7, 16, 1], P, rows, n)
    assert t.tolist() == table and ln.tolist() == length and status.tolist() == st
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.mq_pages_next(pool, t, ln, t, ln, status, add=add, ws=ws)
    for i in range(5):
        graph.replay()
        torch.cuda.synchronize()
        table, length, st, _ = R.next_pages(table, length, None, None, [7, 16, 1], P, rows, n)
        assert t.tolist() == table and ln.tolist() == length and status.tolist() == st
