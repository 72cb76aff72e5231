"""mq_attn_prefix against a plain 64-bit attention: one token and many, ragged and empty caches,
grouped heads, every width and type, layouts and strides, rows past a cache's length that hold
NaN, offsets past 2^31, attention weights, in graphs and on other streams. Every test runs on the library
as it is and on a test build that sends calls of any size to the tensor-core kernel (which the library
keeps for large ones) and row tiles of any prefix side by side."""
import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True, params=["as it is", "tensor cores"])
def _library(request):
    require_gpu()
    own = mq.lib()
    if request.param != "as it is":
        mq._lib = mq._load(B.build_variant("attn_many", ["MQ_FEW_BYTES=0", "MQ_MANY_FROM=1", "MQ_LANES_FROM=0"]))
    yield
    mq._lib = own


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _inside(got, want, bound, what):
    got = got.double()
    assert not torch.isnan(got).any(), f"{what}: NaN"
    same = got == want
    bad = ~same & ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst error / bound " \
        f"{float(((got - want).abs() / bound)[~same].max()):.3g}"


def _case(B, T, Hq, Hkv, D, P, cap, lens, dtype, out_dtype=None, scores=False, seed=0, head_major=False, std=1.5,
          garbage=float("nan")):
    out_dtype = out_dtype or dtype
    q = _rand((B, T, Hq, D), dtype, seed, std)

    def cache(n, rows, s):
        if head_major:
            return [_rand((n, Hkv, rows, D), dtype, seed + s + i).transpose(1, 2) for i in range(2)]
        return [_rand((n, rows, Hkv, D), dtype, seed + s + i) for i in range(2)]

    pk, pv = cache(1, P, 10) if P else (None, None)
    k, v = cache(B, cap, 20) if cap else (None, None)
    n = None
    if cap:
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b in range(B):
            k[b, max(0, min(lens[b], cap)):] = garbage
            v[b, max(0, min(lens[b], cap)):] = garbage
    out = Guarded((B, T, Hq, D), out_dtype)
    lse = Guarded((B, T, Hq), F32)
    score = torch.rand((B, Hkv, cap), device="cuda") if scores else None
    score_out = Guarded((B, Hkv, cap), F32) if scores else None
    mq.mq_attn_prefix(q, mq.KV(pk, pv) if P else None, mq.KV(k, v) if cap else None, n, out.t, lse=lse.t, score=score,
                      score_out=score_out.t if scores else None)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    want, bound = R.attention(q, pk[0] if P else None, pv[0] if P else None, k, v, lens, D ** -0.5, out_dtype, score)
    _inside(out.t, want[0], bound[0], "out")
    _inside(lse.t, want[1], bound[1], "lse")
    out.check()
    lse.check()
    if scores:
        score_out.check()
        for b in range(B):
            m = max(0, min(lens[b], cap))
            _inside(score_out.t[b, :, :m], want[2][b, :, :m], bound[2][b, :, :m], f"score of sequence {b}")
            rest = score_out.t[b, :, m:].contiguous().view(torch.int32)
            assert torch.equal(rest, torch.full_like(rest, -842150451)), "score past the length was written"   # 0xCDCDCDCD
    return out.t


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_decode_widths_and_types(D, dtype):
    _case(3, 1, 10, 2, D, 100, 70, [70, 0, 33], dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (7, 1), (28, 4), (40, 8), (16, 1), (17, 1), (40, 1), (64, 8)])
def test_head_layouts(Hq, Hkv):
    _case(2, 1, Hq, Hkv, 64, 65, 130, [130, 1], F16)


@pytest.mark.parametrize("P", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 640, 3001])
@pytest.mark.parametrize("cap,lens", [(0, None), (1, [1, 0]), (64, [64, 63]), (129, [129, 128]), (700, [65, 700])])
def test_lengths(P, cap, lens):
    if P == 0 and cap == 0:
        pytest.skip("nothing to attend to is its own test")
    _case(2, 1, 4, 2, 128, P, cap, lens or [0, 0], F16, seed=P + cap)


@pytest.mark.parametrize("T", [2, 3, 5, 8, 17, 64, 200, 333])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16), (96, F16)])
def test_several_queries_are_causal(T, D, dtype):
    lens = [T, T + 37, T + 300]
    _case(3, T, 6, 2, D, 150, T + 300, lens, dtype, seed=T)


@pytest.mark.parametrize("P", [0, 70])
def test_queries_that_see_nothing_of_their_own(P):
    """Fewer rows than queries: the first ones see none; without a prefix their output is zero."""
    for T in (4, 130):
        out = _case(3, T, 4, 2, 64, P, T, [0, 1, T - 1], F16)
        if P == 0:
            assert not out[0].any() and not out[1, :T - 1].any()


def test_lengths_outside_the_cache_are_clamped():
    _case(3, 1, 4, 2, 64, 0, 40, [-5, 41, 1 << 30], F16)


def test_an_empty_prefix_and_an_empty_cache():
    q = _rand((2, 1, 4, 64), F16, 1)
    out, lse = torch.full_like(q, 7), torch.zeros((2, 1, 4), device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    mq.mq_attn_prefix(q, mq.KV.empty(1, 0, 2, 64), mq.KV.empty(2, 0, 2, 64), n, out, lse=lse)
    assert not out.any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("B", [1, 9, 33, 70])
def test_batches_on_one_prefix(B):
    """More rows than one tile of any kind; ragged lengths with one long sequence among short ones."""
    lens = [(n * 37) % 90 for n in range(B)]
    lens[B // 2] = 900
    _case(B, 1, 14, 2, 128, 777, 900, lens, BF16)


@pytest.mark.parametrize("out_dtype", [F16, F32])
def test_outputs_in_32_bits(out_dtype):
    _case(2, 1, 8, 2, 128, 300, 90, [90, 17], F16, out_dtype=out_dtype)
    _case(1, 150, 8, 2, 128, 300, 200, [200], F16, out_dtype=out_dtype)


@pytest.mark.parametrize("T", [1, 4, 70])
def test_head_major_layout(T):
    _case(2, T, 8, 4, 128, 200, 150, [150, 71], F16, head_major=True)


@pytest.mark.parametrize("T", [1, 40])
def test_strided_views(T):
    """q as a slice of wider rows, caches as every second row and the upper heads of larger ones."""
    B, Hq, Hkv, D, cap, P = 2, 6, 2, 64, 90, 50
    wide = _rand((B, T, Hq + 4, D), F16, 3)
    q = wide[:, :, 2:2 + Hq]
    big = [_rand((B, 2 * cap, Hkv + 3, D), F16, 4 + i) for i in range(2)]
    k, v = (x[:, ::2, 3:] for x in big)
    pre = [_rand((2, P, Hkv, 2 * D), F16, 8 + i) for i in range(2)]
    pk, pv = (x[1:, :, :, :D] for x in pre)
    n = torch.tensor([cap, 60], dtype=torch.int32, device="cuda")
    out = torch.empty((B, T, Hq, D), dtype=F16, device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, out)
    want, bound = R.attention(q, pk[0], pv[0], k, v, [cap, 60], D ** -0.5, F16)
    _inside(out, want[0], bound[0], "out")


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("Hq,Hkv", [(10, 2), (40, 1), (4, 4)])
def test_attention_weights(T, Hq, Hkv):
    _case(3, T, Hq, Hkv, 64, 45, 333, [333, 0, 100], F16, scores=True)
    _case(2, T, Hq, Hkv, 128, 0, 130, [130, T], BF16, scores=True)


def test_weights_in_place_and_nothing_seen():
    B, Hkv, cap = 2, 2, 40
    q, k, v = _rand((B, 6, 4, 64), F16, 1), _rand((B, cap, Hkv, 64), F16, 2), _rand((B, cap, Hkv, 64), F16, 3)
    n = torch.tensor([3, 40], dtype=torch.int32, device="cuda")   # sequence 0: three queries see nothing
    score = torch.zeros((B, Hkv, cap), device="cuda")
    out = torch.empty((B, 6, 4, 64), dtype=F32, device="cuda")
    for _ in range(2):
        mq.mq_attn_prefix(q, None, mq.KV(k, v), n, out, score=score, score_out=score)
    want, _ = R.attention(q, None, None, k, v, [3, 40], 0.125, F32, torch.zeros_like(score))
    assert float((score.double() - 2 * want[2]).abs().max()) < 1e-4
    # every query that sees a key gives a weight of one in all
    assert abs(float(score[0].sum()) - 2 * 3 * 4) < 1e-3 and abs(float(score[1].sum()) - 2 * 6 * 4) < 1e-3


@pytest.mark.parametrize("T", [1, 130])
def test_large_products(T):
    """Products of thousands: the softmax picks single keys, nothing overflows."""
    _case(2, T, 4, 2, 64, 100, T + 50, [T + 50, T], F16, std=600.0)


@pytest.mark.parametrize("T", [1, 90])
def test_nan_stays_in_its_sequence(T):
    B, cap = 3, 200
    q, k, v = _rand((B, T, 4, 64), F16, 1), _rand((B, cap, 2, 64), F16, 2), _rand((B, cap, 2, 64), F16, 3)
    pk, pv = _rand((1, 50, 2, 64), F16, 4), _rand((1, 50, 2, 64), F16, 5)
    n = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    clean = torch.empty((B, T, 4, 64), dtype=F16, device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, clean)
    k[1, 5, 0] = float("nan")
    v[1, 7, 1] = float("inf")
    out = torch.empty_like(clean)
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, out)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert bool(out[1, -1, :2].isnan().all()) and not bool(out[1, -1, 2:].isfinite().any())


def test_offsets_past_32_bits():
    """Two caches 5 GB apart in one allocation, and rows 17 MB apart."""
    D, Hkv, cap = 64, 2, 300
    raw = torch.empty((2, 2 ** 31 + 2 ** 29), dtype=F16, device="cuda")
    seq, row = 2 ** 31 + 2 ** 28, 8388608
    k = raw[0].as_strided((2, cap, Hkv, D), (seq, Hkv * D, D, 1))
    v = raw[1].as_strided((2, cap, Hkv, D), (seq, Hkv * D, D, 1))
    pk = raw[0][2 ** 20:].as_strided((1, 260, Hkv, D), (0, row, D, 1))
    pv = raw[1][2 ** 20:].as_strided((1, 260, Hkv, D), (0, row, D, 1))
    for i, t in enumerate((k, v, pk, pv)):
        t.copy_(_rand(t.shape, F16, 30 + i))
    for T in (1, 70):
        q = _rand((2, T, 4, D), F16, 40)
        n = torch.tensor([cap, 155], dtype=torch.int32, device="cuda")
        out = torch.empty((2, T, 4, D), dtype=F16, device="cuda")
        mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, out)
        want, bound = R.attention(q, pk[0], pv[0], k, v, [cap, 155], D ** -0.5, F16)
        _inside(out, want[0], bound[0], "out")


@pytest.mark.parametrize("T,scores", [(1, False), (1, True), (5, False), (140, False)])
def test_graph_replays_and_other_streams(T, scores):
    B, Hq, Hkv, D, P, cap = 3, 14, 2, 128, 500, 300
    q, k, v = _rand((B, T, Hq, D), BF16, 1), _rand((B, cap, Hkv, D), BF16, 2), _rand((B, cap, Hkv, D), BF16, 3)
    pre = mq.KV(_rand((1, P, Hkv, D), BF16, 4), _rand((1, P, Hkv, D), BF16, 5))
    n = torch.tensor([300, 150, 222], dtype=torch.int32, device="cuda")
    own = mq.KV(k, v)
    score = torch.rand((B, Hkv, cap), device="cuda") if scores else None
    so = torch.zeros((B, Hkv, cap), device="cuda") if scores else None
    ws = mq.attn_workspace(B, T, Hq, Hkv, D, P, cap, scores)
    out = torch.empty((B, T, Hq, D), dtype=BF16, device="cuda")

    def step(stream=None):
        mq.mq_attn_prefix(q, pre, own, n, out, score=score, score_out=so, ws=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    first, first_so = out.clone(), so.clone() if scores else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([300, 150, 222], [T, 300, 299]):       # lengths change between replays
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        out.zero_()
        if scores:
            so.zero_()                                  # rows past a length are not written
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    n.copy_(torch.tensor([300, 150, 222], dtype=torch.int32))
    if scores:
        so.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and (not scores or torch.equal(so, first_so))


def test_a_workspace_of_garbage_and_one_that_is_too_small():
    B, Hq, Hkv, D, P, cap = 2, 8, 2, 64, 400, 100
    q = _rand((B, 1, Hq, D), F16, 1)
    pre = mq.KV(_rand((1, P, Hkv, D), F16, 4), _rand((1, P, Hkv, D), F16, 5))
    own = mq.KV(_rand((B, cap, Hkv, D), F16, 2), _rand((B, cap, Hkv, D), F16, 3))
    n = torch.tensor([100, 0], dtype=torch.int32, device="cuda")
    need = mq.mq_attn_ws_bytes(B, 1, Hq, Hkv, D, P, cap)
    outs = []
    for fill in (0, 255, 0x7F):
        ws = Guarded((need,), torch.uint8)
        ws.t.fill_(fill)
        out = torch.empty((B, 1, Hq, D), dtype=F16, device="cuda")
        mq.mq_attn_prefix(q, pre, own, n, out, ws=ws.t)
        torch.cuda.synchronize()
        ws.check()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    with pytest.raises(mq.MQError) as e:
        mq.mq_attn_prefix(q, pre, own, n, out, ws=torch.empty((need - 16,), dtype=torch.uint8, device="cuda"))
    assert e.value.status == mq.MQ_ERR_SCRATCH


def test_binding_refuses():
    q = _rand((2, 1, 4, 64), F16, 1)
    own = mq.KV.empty(2, 10, 2, 64)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    for bad in (dict(q=q.bfloat16()), dict(q=q.cpu()), dict(out=out.bfloat16()), dict(own_len=n.long()),
                dict(own_len=n[:1]), dict(out=out[:1]), dict(q=q[..., :32]), dict(own="cache"),
                dict(own=None), dict(lse=torch.empty(3, device="cuda"))):
        a = dict(q=q, prefix=None, own=own, own_len=n, out=out) | bad
        with pytest.raises((TypeError, ValueError)):
            mq.mq_attn_prefix(**a)
    score = torch.zeros((2, 2, 10), device="cuda")
    for bad, status in ((dict(score=score), mq.MQ_ERR_NULL), (dict(scale=float("nan")), mq.MQ_ERR_SHAPE),
                        (dict(prefix=mq.KV.empty(2, 4, 2, 64)), mq.MQ_ERR_SHAPE),
                        (dict(prefix=mq.KV.empty(1, 4, 4, 64)), mq.MQ_ERR_SHAPE),
                        (dict(prefix=mq.KV.empty(1, 4, 2, 64, BF16)), mq.MQ_ERR_TYPE),
                        (dict(own=mq.KV.empty(3, 10, 2, 64), own_len=torch.zeros(3, dtype=torch.int32, device="cuda")),
                         None)):
        a = dict(q=q, prefix=None, own=own, own_len=n, out=out) | bad
        with pytest.raises((mq.MQError, ValueError)) as e:
            mq.mq_attn_prefix(**a)
        if status is not None:
            assert e.value.status == status


@pytest.mark.parametrize("T,P,cap,lens,Hq,Hkv,dtype", [(1500, 700, 1600, [1600], 28, 4, BF16), (700, 0, 700, [700, 650, 699], 32, 8, F16),
                                                      (3314, 1000, 3314, [3314], 28, 4, BF16)])
def test_long_prompts(T, P, cap, lens, Hq, Hkv, dtype):
    """Prompts that the tensor-core kernel takes; sampled queries against the reference, first and last rows of
    tiles among them."""
    B, D = len(lens), 128
    q = _rand((B, T, Hq, D), dtype, 1, 1.5)
    k, v = _rand((B, cap, Hkv, D), dtype, 2), _rand((B, cap, Hkv, D), dtype, 3)
    pk, pv = (_rand((1, P, Hkv, D), dtype, 4 + i) for i in range(2)) if P else (None, None)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("nan")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = torch.empty((B, T, Hq, D), dtype=dtype, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv) if P else None, mq.KV(k, v), n, out, lse=lse)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    assert not out[:, max(0, T - min(lens)):].isnan().any()
    only = [0, 35, 36, 127, 128, 255, 256, T // 2, T - 50, T - 1]
    want, bound = R.attention(q, pk[0] if P else None, pv[0] if P else None, k, v, lens, D ** -0.5, dtype, only=only)
    _inside(out[:, only], want[0][:, only], bound[0][:, only], "out")
    _inside(lse[:, only], want[1][:, only], bound[1][:, only], "lse")


@pytest.mark.parametrize("B,Hq,Hkv,P", [(64, 40, 8, 7000), (33, 28, 4, 13001), (300, 8, 2, 25000)])
def test_long_prefixes_of_large_batches(B, Hq, Hkv, P):
    """Prefixes that several row tiles read side by side, with ragged own caches; sampled sequences."""
    D, cap, dtype = 128, 100, F16
    q, pk, pv = _rand((B, 1, Hq, D), dtype, 1, 1.5), _rand((1, P, Hkv, D), dtype, 2), _rand((1, P, Hkv, D), dtype, 3)
    k, v = _rand((B, cap, Hkv, D), dtype, 4), _rand((B, cap, Hkv, D), dtype, 5)
    lens = [(37 * b) % 101 for b in range(B)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = torch.empty((B, 1, Hq, D), device="cuda"), torch.empty((B, 1, Hq), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, out, lse=lse)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    for b in [0, 1, B // 2, B - 1]:
        want, bound = R.attention(q[b:b + 1], pk[0], pv[0], k[b:b + 1], v[b:b + 1], lens[b:b + 1], D ** -0.5, F32)
        _inside(out[b:b + 1], want[0], bound[0], f"out of {b}")
        _inside(lse[b:b + 1], want[1], bound[1], f"lse of {b}")


def test_scales_of_any_sign():
    for scale in (0.3, -0.2, 0.0):
        for T in (1, 40):
            q, k, v = _rand((1, T, 4, 64), F16, 1), _rand((1, 90, 2, 64), F16, 2), _rand((1, 90, 2, 64), F16, 3)
            n = torch.tensor([77], dtype=torch.int32, device="cuda")
            out = torch.empty((1, T, 4, 64), dtype=F16, device="cuda")
            mq.mq_attn_prefix(q, None, mq.KV(k, v), n, out, scale=scale)
            want, bound = R.attention(q, None, None, k, v, [77], scale, F16)
            _inside(out, want[0], bound[0], f"scale {scale}")


@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (6, 2), (5, 1)])
def test_results_do_not_depend_on_what_ran_before(Hq, Hkv):
    """Row tiles that are not full (groups that do not divide 256): what other calls left in their places must not
    show in the rows beside them, not in the last bit either."""
    T, D, P, cap = 700, 128, 300, 700
    q, k, v = _rand((1, T, Hq, D), BF16, 1), _rand((1, cap, Hkv, D), BF16, 2), _rand((1, cap, Hkv, D), BF16, 3)
    pre = mq.KV(_rand((1, P, Hkv, D), BF16, 4), _rand((1, P, Hkv, D), BF16, 5))
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    own, results = mq.KV(k, v), []
    for std in (0.0, 1.0, 30.0, 300.0):
        full = _rand((1, 2048, 8, D), BF16, 6, std)          # eight heads to a key head: full tiles
        other = mq.KV(_rand((1, 2048, 1, D), BF16, 7), _rand((1, 2048, 1, D), BF16, 8))
        mq.mq_attn_prefix(full, None, other, torch.full((1,), 2048, dtype=torch.int32, device="cuda"),
                          torch.empty_like(full))
        out, lse = torch.empty((1, T, Hq, D), device="cuda"), torch.empty((1, T, Hq), device="cuda")
        mq.mq_attn_prefix(q, pre, own, n, out, lse=lse)
        results.append((out, lse))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])


@pytest.mark.parametrize("T,Hq,Hkv,cap,lens", [(17, 3, 3, 200, [200, 5]), (33, 14, 2, 301, [300, 33]), (150, 7, 1, 404, [404, 20]),
                                                (400, 16, 2, 640, [555, 0]), (5, 28, 4, 1000, [777, 1000])])
def test_score_of_many_queries(T, Hq, Hkv, cap, lens):
    """Weights of several queries' rows added up by one and by several blocks, lengths below and above T, caps that do
    and do not leave every row's products on 16 bytes."""
    _case(2, T, Hq, Hkv, 64, 40, cap, lens, F16, scores=True)
    _case(2, T, Hq, Hkv, 128, 0, cap, lens, BF16, scores=True)
