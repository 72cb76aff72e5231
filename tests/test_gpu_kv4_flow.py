"""The 4-bit cache's calls together, as a serving loop makes them, in lock step with sequences kept as plain lists of rows;
and around them: memory that the binding allocates, calls at the same time, a copy that never comes."""
import ctypes
import math

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as A
from tests import _kv4_ref as R
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu
I32, F16 = torch.int32, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def _rand(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


class Served:
    """Sequences on one pool of two layers, and beside them their rows in 64 bits."""
    LAYERS, HQ, HKV, D, ROWS, WIDTH, PAGES = 2, 8, 2, 128, 16, 12, 60

    def __init__(self):
        self.data = torch.full((self.LAYERS, self.PAGES, mq.mq_kv4_page_bytes(self.ROWS, self.HKV, self.D)), 255, dtype=torch.uint8,
                               device="cuda")
        self.pool = mq.Pool(self.data, self.ROWS)
        self.table, self.length = torch.full((0, self.WIDTH), -1, dtype=I32, device="cuda"), _dev([])
        self.rows = []                                    # [sequence][layer] (keys, values) in 64 bits
        self.seed = 0

    def step(self, frm, keep, add):
        m = len(frm)
        table, length, status = torch.empty((m, self.WIDTH), dtype=I32, device="cuda"), torch.empty((m,), dtype=I32, device="cuda"), _dev([0, 0, 0])
        if not len(self.rows):
            self.table, self.length = torch.full((1, self.WIDTH), -1, dtype=I32, device="cuda"), _dev([0])
        mq.mq_pages_next(self.pool, self.table, self.length, table, length, status, _dev(frm), None if keep is None else _dev(keep), _dev(add))
        self.table, self.length = table, length
        old = self.rows
        nothing = torch.zeros((0, self.HKV, self.D), dtype=torch.float64, device="cuda")
        self.rows = []
        for b, f in enumerate(frm):
            n = None if keep is None else keep[b]
            self.rows.append([tuple(t[:n] for t in old[f][l]) if 0 <= f < len(old) else (nothing, nothing) for l in range(self.LAYERS)])
        assert status.tolist()[0] == 0 and status.tolist()[2] == 0
        # the new rows of every layer, and attention of their tokens
        had = [len(self.rows[b][0][0]) for b in range(m)]
        assert self.length.tolist() == [x + y for x, y in zip(had, add)]
        seq = _dev([b for b in range(m) for _ in range(add[b])])
        row = _dev([had[b] + i for b in range(m) for i in range(add[b])])
        for l in range(self.LAYERS):
            self.seed += 1
            M = len(seq)
            q, k, v = (_rand((M, h, self.D), 10 * self.seed + i) for i, h in enumerate((self.HQ, self.HKV, self.HKV)))
            cache = mq.KV4(self.data[l], self.table, self.ROWS, self.HKV, self.D)
            q16 = torch.empty((M, self.HQ, self.D), dtype=F16, device="cuda")
            mq.mq_qk_norm_rope_kv4(q, k, v, q16, cache, seq, row)
            assert torch.equal(q16, q.half())
            kq, vq = (R.value4(*R.round4(t)) for t in (k, v))
            for b in range(m):
                mine = (seq == b).nonzero()[:, 0]
                self.rows[b][l] = tuple(torch.cat([t, x[mine]]) for t, x in zip(self.rows[b][l], (kq, vq)))
            if len(set(add)) == 1 and add[0]:
                self.attend(l, q16.view(m, add[0], self.HQ, self.D))
            self.read(l)

    def attend(self, l, q):
        m, T = q.shape[:2]
        cache = mq.KV4(self.data[l], self.table, self.ROWS, self.HKV, self.D)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        mq.mq_attn_kv4(q, cache, self.length, out, lse=lse)
        for b in range(m):
            k, v = self.rows[b][l]
            want, bound = A.attention(q[b:b + 1], None, None, k[None], v[None], [len(k)], self.D ** -0.5, F16)
            assert bool(((out[b:b + 1].double() - want[0]).abs() <= bound[0]).all())
            assert bool(((lse[b:b + 1].double() - want[1]).abs() <= bound[1]).all())
        return out

    def read(self, l):
        m = len(self.rows)
        kv = mq.KV.empty(m, self.WIDTH * self.ROWS, self.HKV, self.D, torch.bfloat16)
        mq.mq_kv4_read(mq.KV4(self.data[l], self.table, self.ROWS, self.HKV, self.D), self.length, kv)
        for b in range(m):
            for got, want in zip((kv.k, kv.v), self.rows[b][l]):
                assert torch.equal(got[b, :len(want)].double(), want)

    def compact(self):
        out = torch.empty_like(self.table)
        where, live = torch.empty((self.PAGES,), dtype=I32, device="cuda"), _dev([0])
        mq.mq_pages_compact(self.pool, self.table, self.length, out, where, live)
        used = sorted({p for row, n in zip(self.table.tolist(), self.length.tolist()) for p in row[:-(-n // self.ROWS)]})
        assert live.item() == len(used) and int(out.max()) < len(used)
        self.table = out
        self.data[:, len(used):] = 255                     # what is left is nobody's
        for l in range(self.LAYERS):
            self.read(l)


def test_serving_loop():
    s = Served()
    s.step([-1, -1, -1], None, [37, 37, 37])               # three prompts
    s.step([0, 1, 2], None, [1, 1, 1])
    s.step([0, 0, 0, 1, 2, 2], None, [1] * 6)              # forked in the middle of a page
    s.step([0, 1, 2, 3, 4, 5], [36, 39, 38, 30, 16, 39], [5] * 6)    # trimmed, five drafted tokens each
    s.step([5, 3, 1, 1], [40, 31, 44, 41], [2, 0, 3, 1])   # two sequences end, two go on from one
    s.compact()
    s.step([0, 1, 2, 3, -1], None, [1] * 5)
    q = _rand((5, 1, s.HQ, s.D), 99).half()
    before = [s.attend(l, q) for l in range(s.LAYERS)]
    s.compact()
    assert all(torch.equal(a, s.attend(l, q)) for l, a in enumerate(before))
    s.step([4, 3], None, [16, 20])
    s.step([0, 1, 0, 1], None, [1] * 4)
    assert mq.mq_device_status() == mq.MQ_OK


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("T", [1, 70])
def test_attention_with_a_workspace_of_its_own(T, raw):
    """What the binding allocates for a call on another stream must not meet what the current one allocates next."""
    n, Hq, Hkv, D = 3, 8, 2, 128
    cache = R.random_cache(n, 12, 64, Hkv, D, 7)
    length = _dev([700, 650, 75])
    q = _rand((n, T, Hq, D), 1).half()
    want = torch.empty_like(q)
    mq.mq_attn_kv4(q, cache, length, want, ws=mq.attn_kv4_workspace(n, T, Hq, Hkv, D, cache.cap))
    size = mq.mq_attn_kv4_ws_bytes(n, T, Hq, Hkv, D, cache.cap)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)                     # about a ms: the kernels run after what follows here
        mq.mq_attn_kv4(q, cache, length, out, stream=side.cuda_stream if raw else side)
        other = [torch.full((size,), i, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(bool((x == i).all()) for x in other)


def test_pages_with_a_workspace_of_their_own():
    r, width, P = 16, 6, 40
    data = torch.zeros((1, P, 64), dtype=torch.uint8, device="cuda")
    pool = mq.Pool(data, r)
    table, length = [[0, 1, 2, -1, -1, -1], [3, -1, -1, -1, -1, -1]], [40, 5]
    want = R.next_pages(table, length, [0, 0, 1], None, [9, 9, 30], P, r, 3)
    side = torch.cuda.Stream()
    t, n, frm, add = _dev(table), _dev(length), _dev([0, 0, 1]), _dev([9, 9, 30])
    size = mq.mq_pages_ws_bytes(pool, 3, width)
    for i in range(5):
        t_out, n_out, status = torch.zeros((3, width), dtype=I32, device="cuda"), _dev([0] * 3), _dev([0] * 3)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)
        mq.mq_pages_next(pool, t, n, t_out, n_out, status, frm, None, add, stream=side)
        other = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert t_out.tolist() == want[0] and n_out.tolist() == want[1] and status.tolist() == want[2]
        assert all(bool((x == 255).all()) for x in other)


def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    Hq, Hkv, D = 8, 2, 128
    jobs = []
    for i, (n, T) in enumerate(((4, 1), (2, 5))):
        cache = R.random_cache(n, 30, 32, Hkv, D, 30 + i)
        q, length = _rand((n, T, Hq, D), i).half(), _dev([900 - 100 * j for j in range(n)])
        jobs.append((q, cache, length, torch.empty_like(q), mq.attn_kv4_workspace(n, T, Hq, Hkv, D, cache.cap), torch.cuda.Stream()))
    want = []
    for q, cache, length, out, ws, _ in jobs:
        mq.mq_attn_kv4(q, cache, length, out, ws=ws)
        want.append(out.clone())
    torch.cuda.synchronize()
    for _ in range(20):
        for q, cache, length, out, ws, s in jobs:
            mq.mq_attn_kv4(q, cache, length, out, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(job[3], w) for job, w in zip(jobs, want))


def test_wait_runs_out_is_reported_and_forgotten():
    """A test build (50 ms wait limit) whose first block leaves out a copy: the call returns, the status says so once, and the
    next call is right."""
    own = mq.lib()
    L = mq._load(B.build_variant("kv4_split", ["MQ_KV4_SPLIT_FROM=0", "MQ_TEST_INJECT", "MQ_WAIT_LIMIT_NS=50000000ull"]))
    L.mq_test_inject_kv4.restype, L.mq_test_inject_kv4.argtypes = ctypes.c_int, [ctypes.c_int]
    mq._lib = L
    try:
        n, Hq, Hkv, D = 2, 8, 2, 128
        cache = R.random_cache(n, 20, 32, Hkv, D, 3)
        q, length = _rand((n, 1, Hq, D), 4).half(), _dev([600, 333])
        out, ws = torch.zeros_like(q), mq.attn_kv4_workspace(n, 1, Hq, Hkv, D, cache.cap)
        ws.fill_(0x7F)                                     # entries that are not written must not be followed
        assert mq.mq_device_status() == mq.MQ_OK
        assert L.mq_test_inject_kv4(1) == mq.MQ_OK
        mq.mq_attn_kv4(q, cache, length, out, ws=ws)
        torch.cuda.synchronize()
        assert mq.mq_device_status() == mq.MQ_ERR_DEVICE
        assert mq.mq_device_status() == mq.MQ_OK
        assert L.mq_test_inject_kv4(0) == mq.MQ_OK
        mq.mq_attn_kv4(q, cache, length, out, ws=ws)
        torch.cuda.synchronize()
        assert mq.mq_device_status() == mq.MQ_OK
        k, v = R.gather(cache.pages, cache.table, 32, Hkv, D, [600, 333])
        want, bound = A.attention(q, None, None, k, v, [600, 333], D ** -0.5, F16)
        assert bool(((out.double() - want[0]).abs() <= bound[0]).all())
    finally:
        L.mq_test_inject_kv4(0)
        mq._lib = own


@pytest.mark.parametrize("T", [1, 5, 70])
def test_tables_and_pools_of_nothing(T):
    """Tables without entries, pools without pages: queries are there all the same."""
    n, Hq, H, D, rows = 2, 8, 2, 64, 16
    q = torch.randn((n, T, Hq, D), device="cuda").to(F16)
    none = torch.empty((n, 0), dtype=I32, device="cuda")
    holes = torch.full((n, 5), -1, dtype=I32, device="cuda")
    size = mq.mq_kv4_page_bytes(rows, H, D)
    some, empty = torch.zeros((3, size), dtype=torch.uint8, device="cuda"), torch.empty((0, size), dtype=torch.uint8, device="cuda")
    length = torch.tensor([77, 80], dtype=I32, device="cuda")
    for cache, seen in ((mq.KV4(some, none, rows, H, D), 0), (mq.KV4(empty, none, rows, H, D), 0), (mq.KV4(empty, holes, rows, H, D), 77)):
        out, lse = torch.full_like(q, 3.0), torch.zeros((n, T, Hq), device="cuda")
        mq.mq_attn_kv4(q, cache, length, out, lse=lse)
        assert (out == 0).all()
        for b in range(n):
            for t in range(T):
                k = max(0, min(int(length[b]), cache.cap) - T + 1 + t)       # all keys are zeros
                want = math.log(k) if k else -math.inf       # (log(128 k) - 7 log 2, a rounding or two of 2^-24 of each)
                assert all(x == want or abs(x - want) <= 2e-6 * abs(want) + 2e-6 for x in lse[b, t].tolist())
        x, q_out = torch.randn((4, Hq, D), device="cuda"), torch.zeros((4, Hq, D), dtype=F16, device="cuda")
        k = torch.randn((4, H, D), device="cuda")
        row = torch.arange(4, dtype=I32, device="cuda")
        mq.mq_qk_norm_rope_kv4(x, k, k, q_out, cache, None, row)
        assert torch.equal(q_out, x.to(F16))
        kv = mq.KV.empty(n, 96, H, D)
        kv.k.fill_(7.0)
        kv.v.fill_(7.0)
        mq.mq_kv4_read(cache, length, kv)
        for b in range(n):
            m = min(int(length[b]), cache.cap)
            for y in (kv.k[b], kv.v[b]):
                assert (y[:m] == 0).all() and (y[m:] == 7).all()
    assert (some == 0).all()
    assert mq.mq_device_status() == mq.MQ_OK


def test_pages_of_nothing():
    status, live = torch.full((3,), 9, dtype=I32, device="cuda"), torch.full((1,), 9, dtype=I32, device="cuda")

    def ints(*x):
        return torch.tensor(x, dtype=I32, device="cuda")

    def table(n, width):
        return torch.full((n, width), 77, dtype=I32, device="cuda")

    pool = mq.Pool(torch.zeros((2, 6, 32), dtype=torch.uint8, device="cuda"), 16)
    # from no sequences
    out, length = table(2, 3), ints(5, 5)
    mq.mq_pages_next(pool, table(0, 3), ints(), out, length, status, ints(0, -1), None, ints(17, 0))
    assert (out.tolist(), length.tolist(), status.tolist()) == ([[0, 1, -1], [-1, -1, -1]], [17, 0], [0, 4, 0])
    # to none
    mq.mq_pages_next(pool, out, length, table(0, 3), ints(), status, ints(), None, None)
    assert status.tolist() == [0, 6, 0]
    # tables without entries
    mq.mq_pages_next(pool, table(2, 0), ints(4, 4), table(2, 0), length, status, None, None, ints(1, 0))
    assert (length.tolist(), status.tolist()) == ([0, 0], [0, 6, 1])
    # no pages
    bare = mq.Pool(torch.zeros((2, 0, 32), dtype=torch.uint8, device="cuda"), 16)
    out, length = table(2, 3), ints(0, 0)
    mq.mq_pages_next(bare, table(2, 3), ints(0, 0), out, length, status, None, None, ints(1, 0))
    assert (out.tolist(), length.tolist(), status.tolist()) == ([[-1] * 3] * 2, [0, 0], [1, 0, 0])
    mq.mq_pages_compact(bare, out, length, out, ints(), live)
    assert live.tolist() == [0]
    where = torch.full((6,), 9, dtype=I32, device="cuda")
    mq.mq_pages_compact(pool, table(0, 3), ints(), table(0, 3), where, live)
    assert (where.tolist(), live.tolist()) == ([-1] * 6, [0])
