"""mq_qk_norm_rope and mq_kv_evict against plain 64-bit forms: widths, pairings, axes, positions of any
size, slots, strides; ties, NaN, lengths at and around the budget, in place and apart."""
import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rand(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def _inside(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def _rope_case(M, Hq, Hkv, D, n, dtype, n_axes=1, inter=False, norm=True, pos=None, slot=None, cap=None, seed=0,
               head_major=False):
    q, kv = _rand((M, Hq, D), seed), _rand((M, 2 * Hkv, D), seed + 1, 3.0)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    wq, wk = (_rand((D,), seed + 2, 0.2) + 1, _rand((D,), seed + 3, 0.2) + 1) if norm else (None, None)
    freq = mq.rope_freq(n) if n else None
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if pos is None:
        pos = torch.randint(0, 40000, (n_axes, M), generator=g, device="cuda", dtype=torch.int32)
    axis = torch.randint(0, n_axes, (n,), generator=g, device="cuda", dtype=torch.uint8) if n_axes > 1 else None
    cap = cap or M
    qo = Guarded((M, Hq, D), dtype)
    shape = (2, Hkv, cap, D) if head_major else (2, cap, Hkv, D)
    kc, vc = Guarded(shape, dtype), Guarded(shape, dtype)
    view = (lambda t: t.transpose(1, 2)) if head_major else (lambda t: t)
    before = view(kc.t).clone()
    mq.mq_qk_norm_rope(q, k, v, qo.t, mq.KV(view(kc.t), view(vc.t)), slot, pos if n else None, freq, axis, wq, wk, 1e-6,
                       inter)
    torch.cuda.synchronize()
    for x in (qo, kc, vc):
        x.check()
    want, bound = R.rope(q, wq, 1e-6, pos, freq, axis, n_axes, inter, dtype)
    _inside(qo.t, want, bound, "q")
    want, bound = R.rope(k, wk, 1e-6, pos, freq, axis, n_axes, inter, dtype)
    slots = list(range(M)) if slot is None else slot.tolist()
    live = [m for m in range(M) if 0 <= slots[m] < 2 * cap]
    got_k, got_v = view(kc.t).reshape(2 * cap, Hkv, D), view(vc.t).reshape(2 * cap, Hkv, D)
    at = [slots[m] for m in live]
    _inside(got_k[at], want[live], bound[live], "k")
    assert torch.equal(got_v[at], v.to(dtype)[live])
    rest = [r for r in range(2 * cap) if r not in set(at)]
    assert torch.equal(got_k[rest].view(torch.int16), before.reshape(2 * cap, Hkv, D)[rest].view(torch.int16))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,n", [(8, 4), (8, 0), (16, 3), (64, 32), (64, 16), (80, 10), (80, 40), (96, 48), (96, 44), (128, 64),
                                 (128, 1), (128, 0), (136, 68), (192, 96), (256, 128), (256, 61)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_widths_and_pairings(D, n, inter, dtype):
    _rope_case(5, 3, 2, D, n, dtype, inter=inter)
    _rope_case(3, 5, 1, D, n, dtype, inter=inter, norm=False)


@pytest.mark.parametrize("M", [1, 2, 7, 100, 1300, 5000])
def test_rope_tokens_and_head_counts(M):
    _rope_case(M, 28, 4, 128, 64, BF16, n_axes=3, seed=M)
    _rope_case(M, 1, 1, 64, 32, F16, seed=M)


def test_rope_positions_of_any_size():
    pos = torch.tensor([[0, 1, -1, 100000, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), 123456789]],
                       dtype=torch.int32, device="cuda")
    _rope_case(9, 4, 2, 128, 64, F16, pos=pos)
    _rope_case(9, 4, 2, 128, 64, F16, pos=pos, inter=True, norm=False)


def test_rope_axis_past_the_last_counts_as_the_last():
    M, D, n = 4, 64, 32
    q = _rand((M, 2, D), 1)
    pos = torch.tensor([[1, 2, 3, 4], [50, 60, 70, 80]], dtype=torch.int32, device="cuda")
    outs = []
    for a in (1, 200):
        o = torch.empty((M, 2, D), dtype=F16, device="cuda")
        mq.mq_qk_norm_rope(q, None, None, o, mq.KV.empty(1, 0, 2, D), None, pos, mq.rope_freq(n),
                           torch.full((n,), a, dtype=torch.uint8, device="cuda"))
        outs.append(o)
    assert torch.equal(outs[0], outs[1])


def test_rope_sections_helper():
    assert mq.rope_axes((2, 1, 3)).tolist() == [0, 0, 1, 2, 2, 2]


@pytest.mark.parametrize("head_major", [False, True])
def test_rope_slots(head_major):
    """Scattered rows of two sequences, padding tokens, slots outside the cache."""
    slot = torch.tensor([5, -1, 9, 0, 10, 2147483647, -2147483648, 3, 20], dtype=torch.int32, device="cuda")
    _rope_case(9, 4, 2, 64, 32, F16, slot=slot, cap=5, head_major=head_major)


def test_rope_parts_alone_and_zero_rows():
    M, D = 6, 64
    x = _rand((M, 2, D), 1)
    x[2] = 0                                           # a row of zeros: the norm gives zeros, not NaN
    kv = mq.KV(torch.zeros((1, M, 2, D), dtype=F16, device="cuda"), torch.zeros((1, M, 2, D), dtype=F16, device="cuda"))
    w = torch.ones(D, device="cuda")
    mq.mq_qk_norm_rope(None, x, None, None, kv, wk=w)
    want, bound = R.rope(x, w, 1e-6, None, None, None, 0, False, F16)
    _inside(kv.k[0], want, bound, "k alone")
    assert not kv.k[0, 2].any() and not kv.v.any()
    mq.mq_qk_norm_rope(None, None, x, None, kv)
    assert torch.equal(kv.v[0], x.half())
    mq.mq_qk_norm_rope(x[:0], None, None, torch.empty((0, 2, D), dtype=F16, device="cuda"), kv)   # M == 0
    x[1, 0, 3] = float("nan")                          # stays in its head
    o = torch.empty((M, 2, D), dtype=F16, device="cuda")
    mq.mq_qk_norm_rope(x, None, None, o, kv, wq=w)
    assert bool(o[1, 0].isnan().all()) and int(o.isnan().sum()) == D


def test_rope_cache_past_32_bits():
    D, H = 64, 2
    raw = torch.empty((2, 2 ** 31 + 2 ** 22), dtype=F16, device="cuda")
    k, v = (raw[i].as_strided((2, 3, H, D), (2 ** 31 + 2 ** 20, H * D, D, 1)) for i in range(2))
    x = _rand((2, H, D), 1)
    slot = torch.tensor([1, 5], dtype=torch.int32, device="cuda")
    mq.mq_qk_norm_rope(None, x, x, None, mq.KV(k, v), slot)
    assert torch.equal(k[0, 1], x[0].half()) and torch.equal(v[1, 2], x[1].half())


def test_rope_binding_refuses():
    q, kv = _rand((2, 4, 64), 1), mq.KV.empty(1, 4, 2, 64)
    out = torch.empty((2, 4, 64), dtype=F16, device="cuda")
    pos, f = torch.zeros(2, dtype=torch.int32, device="cuda"), mq.rope_freq(32)
    ok = dict(q=q, k=None, v=None, q_out=out, cache=kv, pos=pos, inv_freq=f)
    mq.mq_qk_norm_rope(**ok)
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(q_out=out.bfloat16()), dict(q_out=out[:1]), dict(pos=pos.long()),
                dict(pos=pos[:1]), dict(q=None), dict(k=_rand((2, 3, 64), 1)), dict(q=q.transpose(0, 1)),
                dict(wq=torch.ones(63, device="cuda")), dict(axis=torch.zeros(31, dtype=torch.uint8, device="cuda")),
                dict(slot=pos[:1])):
        with pytest.raises((TypeError, ValueError)):
            mq.mq_qk_norm_rope(**(ok | bad))
    for bad, status in ((dict(inv_freq=mq.rope_freq(33)), mq.MQ_ERR_SHAPE),
                        (dict(pos=torch.zeros((9, 2), dtype=torch.int32, device="cuda")), mq.MQ_ERR_SHAPE),
                        (dict(k=_rand((2, 2, 64), 1), cache=mq.KV.empty(1, 1, 2, 64)), mq.MQ_ERR_SHAPE)):
        with pytest.raises(mq.MQError) as e:
            mq.mq_qk_norm_rope(**(ok | bad))
        assert e.value.status == status


# ------------------------------------------------------------------------------------------- eviction

def _evict_case(n, H, D, cap, lens, keep, recent, dst_cap=None, dtype=F16, seed=0, kind="skew", in_place=False,
                head_major=False, score_in_place=False, no_score_out=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    score = torch.rand((n, H, cap), generator=g, device="cuda")
    if kind == "skew":
        score = score.pow(6)
    elif kind == "ties":
        score = (score * 4).floor()
    elif kind == "equal":
        score = torch.full_like(score, 0.25)
    elif kind == "odd":                                  # zeros of both signs, infinities, NaN, negatives
        pick = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-42, -1e-42, -3.0, 3.0],
                            device="cuda")
        score = pick[torch.randint(0, 9, (n, H, cap), generator=g, device="cuda")]
    dst_cap = cap if in_place else keep if dst_cap is None else dst_cap
    shape = (n, H, cap, D) if head_major else (n, cap, H, D)
    dshape = (n, H, dst_cap, D) if head_major else (n, dst_cap, H, D)
    view = (lambda t: t.transpose(1, 2)) if head_major else (lambda t: t)
    k, v = (_rand(shape, seed + 1 + i).to(dtype) for i in range(2))
    src = mq.KV(view(k), view(v))
    want_k, want_v, want_s = view(k).clone(), view(v).clone(), score.clone()
    if in_place:
        dk, dv, dst = None, None, src
    else:
        dk, dv = Guarded(dshape, dtype), Guarded(dshape, dtype)
        dst = mq.KV(view(dk.t), view(dv.t))
    index = Guarded((n, H, dst_cap), torch.int32)
    so = score if score_in_place else None if no_score_out else torch.full((n, H, dst_cap), 7.0, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mq.mq_kv_evict(src, length, score, keep, recent, dst, length, so, index.t)
    torch.cuda.synchronize()
    index.check()
    for x in (dk, dv):
        if x is not None:
            x.check()
    for b in range(n):
        L = min(max(lens[b], 0), cap)
        assert int(length[b]) == min(L, keep)
        for h in range(H):
            rows = R.evict(want_s[b, h].tolist(), L, keep, recent)
            m = len(rows)
            assert index.t[b, h].tolist() == rows + [-1] * (dst_cap - m), (b, h)
            assert torch.equal(dst.k[b, :m, h], want_k[b, rows, h]) and torch.equal(dst.v[b, :m, h], want_v[b, rows, h])
            if in_place:
                assert torch.equal(dst.k[b, m:, h], want_k[b, m:, h])
            if so is not None:
                assert torch.equal(so[b, h, :m].view(torch.int32), want_s[b, h, rows].view(torch.int32))
                assert not so[b, h, m:].any()


@pytest.mark.parametrize("kind", ["skew", "ties", "equal", "odd"])
@pytest.mark.parametrize("cap,keep,recent", [(64, 16, 4), (1000, 333, 50), (5000, 1024, 1), (5000, 4999, 0), (300, 100, 100)])
def test_evict_selection(cap, keep, recent, kind):
    _evict_case(2, 3, 64, cap, [cap, cap - 17], keep, recent, kind=kind, seed=cap)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,recent", [(0, 0), (1, 0), (1, 1), (40, 7), (64, 64)])
def test_evict_lengths_around_the_budget(keep, recent, in_place):
    lens = [0, 1, keep - 1, keep, keep + 1, 64, 65, -3]
    _evict_case(8, 2, 64, 64, lens, keep, recent, dst_cap=max(keep, 1) + 3, in_place=in_place)


@pytest.mark.parametrize("D", [8, 64, 96, 128, 256])
@pytest.mark.parametrize("in_place,head_major", [(False, False), (True, False), (False, True), (True, True)])
def test_evict_widths_and_layouts(D, in_place, head_major):
    _evict_case(2, 3, D, 700, [700, 650], 211, 30, in_place=in_place, head_major=head_major, dtype=BF16)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_scores_in_place(in_place):
    _evict_case(2, 2, 64, 2000, [2000, 1500], 700, 64, dst_cap=2000, in_place=in_place, score_in_place=True)


def test_evict_without_scores_out():
    _evict_case(1, 2, 64, 100, [100], 30, 3, no_score_out=True)
    _evict_case(1, 2, 64, 100, [100], 30, 3, no_score_out=True, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long(in_place):
    _evict_case(1, 2, 64, 70001, [70001], 20011, 999, in_place=in_place)
    _evict_case(1, 1, 8, 200000, [199999], 150000, 5, in_place=in_place, kind="ties")


@pytest.mark.parametrize("n,H,cap,keep,recent,kind", [
    (1, 1, 4097, 100, 7, "skew"), (1, 2, 40000, 3000, 17, "equal"), (2, 2, 33000, 32999, 1, "odd"),
    (1, 1, 700000, 5000, 100, "skew"), (130, 1, 300, 64, 9, "skew"), (20, 8, 513, 200, 31, "ties"),
    (52, 2, 1000, 1, 0, "odd")])
def test_evict_row_counts_and_stretches(n, H, cap, keep, recent, kind):
    """Few long rows (clusters of blocks, stretches that do and do not fit shared memory), many short ones
    (blocks that move their own rows), length_out the same array as length."""
    _evict_case(n, H, 8, cap, [cap - 3 * (b % 5) for b in range(n)], keep, recent, kind=kind, seed=n)


def test_evict_length_out_apart():
    for n in (2, 60):
        src, dst = mq.KV(*(_rand((n, 90, 2, 64), i).half() for i in range(2))), mq.KV.empty(n, 40, 2, 64)
        length = torch.tensor([90 - b for b in range(n)], dtype=torch.int32, device="cuda")
        out = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        score, index = torch.rand((n, 2, 90), device="cuda"), torch.empty((n, 2, 40), dtype=torch.int32, device="cuda")
        mq.mq_kv_evict(src, length, score, 40, 4, dst, out, None, index)
        assert out.tolist() == [min(90 - b, 40) for b in range(n)] and length.tolist() == [90 - b for b in range(n)]


def test_evict_cache_past_32_bits():
    D, H, cap = 64, 2, 50
    raw = torch.empty((2, 2 ** 31 + 2 ** 22), dtype=F16, device="cuda")
    k, v = (raw[i].as_strided((2, cap, H, D), (2 ** 31 + 2 ** 20, H * D, D, 1)) for i in range(2))
    k.copy_(_rand(k.shape, 1))
    v.copy_(_rand(v.shape, 2))
    score = torch.rand((2, H, cap), device="cuda")
    n = torch.tensor([50, 50], dtype=torch.int32, device="cuda")
    index = torch.empty((2, H, 20), dtype=torch.int32, device="cuda")
    dst = mq.KV.empty(2, 20, H, D)
    no = torch.empty_like(n)
    mq.mq_kv_evict(mq.KV(k, v), n, score, 20, 5, dst, no, None, index)
    for b in range(2):
        for h in range(H):
            rows = R.evict(score[b, h].tolist(), 50, 20, 5)
            assert torch.equal(dst.k[b, :, h], k[b, rows, h]) and torch.equal(dst.v[b, :, h], v[b, rows, h])


def test_evict_refuses():
    src, dst = mq.KV.empty(2, 50, 2, 64), mq.KV.empty(2, 20, 2, 64)
    n = torch.tensor([50, 50], dtype=torch.int32, device="cuda")
    score, so = torch.rand((2, 2, 50), device="cuda"), torch.empty((2, 2, 20), device="cuda")
    index = torch.empty((2, 2, 20), dtype=torch.int32, device="cuda")
    ok = dict(src=src, length=n, score=score, keep=20, recent=5, dst=dst, length_out=n, score_out=so, index=index)
    half = mq.KV(src.k[:, :20], src.v[:, :20])                      # overlaps src without being it
    for bad, status in ((dict(keep=21), mq.MQ_ERR_SHAPE), (dict(recent=21), mq.MQ_ERR_SHAPE),
                        (dict(recent=-1), mq.MQ_ERR_SHAPE), (dict(dst=half), mq.MQ_ERR_SHAPE),
                        (dict(dst=mq.KV.empty(2, 20, 2, 64, BF16)), mq.MQ_ERR_TYPE),
                        (dict(dst=mq.KV.empty(2, 20, 2, 128)), mq.MQ_ERR_SHAPE),
                        (dict(score_out=score), mq.MQ_ERR_SHAPE)):
        with pytest.raises(mq.MQError) as e:
            mq.mq_kv_evict(**(ok | bad))
        assert e.value.status == status, bad
    for bad in (dict(length=n.long()), dict(length=n[:1]), dict(score=score.half()), dict(index=index.long()),
                dict(index=index[:1]), dict(src="cache"), dict(score=score[:1])):
        with pytest.raises((TypeError, ValueError)):
            mq.mq_kv_evict(**(ok | bad))


@pytest.mark.parametrize("cap", [1500, 3000, 9000])
@pytest.mark.parametrize("shared", [1, 2, 127, 128, 129, 300, 511, 512, 513, 1100])
@pytest.mark.parametrize("digits", [8, 16, 24])
def test_evict_scores_that_share_digits(cap, shared, digits):
    """`shared` rows whose scores agree in their first `digits` bits, of which some are kept, among rows far above
    and far below them: one block of 256 and of 1024 threads, and a cluster."""
    g = torch.Generator().manual_seed(shared * 31 + digits)
    above, keep = 100, 100 + (shared + 1) // 2
    low = torch.randint(0, 1 << min(32 - digits, 20), (shared,), generator=g)
    if shared > 4:
        low[::5] = low[0]                               # ties across the border too
    bits = torch.randint(1, 1000, (cap,), generator=g)                       # next to nothing
    place = torch.randperm(cap, generator=g)
    bits[place[:shared]] = 0x3F000000 + low
    bits[place[shared:shared + above]] = 0x41000000 + torch.randint(0, 5000, (above,), generator=g)
    score = bits.to(torch.int32).view(torch.float32).view(1, 1, cap)
    src, dst = mq.KV(*(_rand((1, cap, 1, 8), i).half() for i in range(2))), mq.KV.empty(1, keep, 1, 8)
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    index = torch.empty((1, 1, keep), dtype=torch.int32, device="cuda")
    mq.mq_kv_evict(src, n, score.cuda(), keep, 0, dst, torch.empty_like(n), None, index)
    assert index.view(-1).tolist() == R.evict(score.view(-1).tolist(), cap, keep, 0)
