"""Numbers at the ends of what 32 bits hold, and past them: keys and values that are not finite, written to 4-bit caches, byte for byte;
norms of queries of any size."""
import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as A
from tests import _kv4_ref as R
from tests._gpu_util import require_gpu
from tests.test_gpu_kv4 import _fill_case, _rand, _rope64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("n_pairs,norm,inter", [(0, False, False), (32, False, False), (20, False, True), (64, False, True), (0, True, False)])
def test_infinities(n_pairs, norm, inter):
    """An infinity is written as 7 d of the largest scale, with its sign; what lies past that as well. (A head that is normed or
    turned with one has numbers of no value: only values there.)"""
    M, H, D = 40, 2, 128
    x = _rand((M, 2 * H, D), 17, 40.0)
    at = slice(None) if not norm and n_pairs == 0 else slice(H, None)
    y = x[:, at]
    y[3, 0, 5], y[3, 0, 6], y[4, 1, 127], y[5, 0, 0] = INF, -INF, INF, -INF
    y[6, 0, ::2], y[6, 0, 1::2] = INF, -INF
    y[7, 0, 33], y[7, 1, 64], y[8, 0, 1] = 3.4e38, -3.4e38, 3361.0
    y[9, 1] = INF
    _fill_case(M, 3, H, D, 16, 2, n_pairs, norm=norm, inter=inter, x=x)


def _pages(k, v, D, inter=False, n_pairs=0, wk=None, eps=1e-6):
    """What is written of keys and values [M, H, D], and the plain form's bytes, NaN taken as 0."""
    M, H = k.shape[:2]
    rows = -(-M // 16) * 16
    cache = mq.KV4.empty(1, rows // 16, rows // 16, H, D, 16)
    cache.table.copy_(torch.arange(rows // 16, dtype=torch.int32, device="cuda").view(1, -1))
    nothing = torch.zeros((rows - M, H, D), device="cuda")
    row = torch.arange(M, dtype=torch.int32, device="cuda")
    all_rows = torch.arange(rows, dtype=torch.int32, device="cuda")
    mq.mq_qk_norm_rope_kv4(None, torch.zeros((rows, H, D), device="cuda"), torch.zeros((rows, H, D), device="cuda"), None, cache, None, all_rows)
    pos, freq = row + 11, mq.rope_freq(n_pairs, device="cuda") if n_pairs else None
    mq.mq_qk_norm_rope_kv4(None, k, v, None, cache, None, row, pos, freq, wk=wk, eps=eps, interleaved=inter)
    y = _rope64(k, wk, float(torch.tensor(eps)), pos[None], freq, None, 1, inter, 1.0)
    want = R.pack(*(tuple(t.view(rows // 16, 16, H, -1) for t in R.round4(torch.cat([x.double().nan_to_num(0.0, INF, -INF), nothing.double()])))
                    for x in (y, v)))
    return cache.pages, want


@pytest.mark.parametrize("n_pairs,norm,inter", [(0, False, False), (64, False, False), (50, False, True), (31, True, False), (64, True, True)])
def test_nan_is_written_as_zero(n_pairs, norm, inter):
    """A number of no value is 0 and leaves its neighbours and their scale as they are; a head normed with one is all zeros."""
    M, H, D = 37, 3, 128
    k, v = _rand((M, H, D), 21), _rand((M, H, D), 22)
    k[30, 0, 3] = INF                                  # (normed: infinity over infinity, and zeros)
    for x in (k, v):
        x[0, 0, 0], x[1, 1, 127], x[2, 2, 33:36] = NAN, NAN, -NAN
        x[3, 0, 32:64] = NAN                           # a whole block
        x[4] = NAN
        x[5, 1, ::7], x[5, 1, 1::7] = NAN, 1e5         # beside numbers past the largest scale
        x[6, 0, 0:32:2], x[6, 0, 1:32:2] = NAN, 0.0
        x[7, 2, 8], x[7, 2, 9] = NAN, -3.0
        x[8, 0, 4], x[8, 0, 5], x[8, 0, 6] = NAN, INF, -INF
    got, want = _pages(k, v, D, inter, n_pairs, (_rand((D,), 23, 0.1) + 1) if norm else None)
    assert torch.equal(got, want)


def test_nan_bits():
    """NaN of either sign and any bits."""
    M, H, D = 64, 1, 64
    k, v = (_rand((M, H, D), 31 + i) for i in range(2))
    for x in (k, v):
        bits = x.view(torch.int32)
        for m in range(M):
            bits[m, 0, (7 * m) % D] = (0x7f800001 + 131 * m) if m % 2 else -1 - 4097 * m
    got, want = _pages(k, v, D)
    assert torch.equal(got, want)


@pytest.mark.parametrize("D,inter,n_pairs", [(64, False, 32), (128, False, 64), (128, True, 30), (96, False, 11), (256, True, 128)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-33])
def test_queries_normed_of_any_size(D, inter, n_pairs, dtype, eps):
    """Queries whose mean square 32 bits do not hold, among ones whose it is, keys between them in a warp; an infinity and a NaN make no
    number of their own head alone."""
    M, Hq, Hkv = 26, 5, 2
    size = (10.0 ** torch.linspace(-37, 38, M, device="cuda", dtype=torch.float64))[:, None, None]
    q, k = ((_rand((M, h, D), 41 + h).double().clamp(-3.0, 3.0) * size.roll(h, 0)).float() for h in (Hq, Hkv))
    q[1, 2], q[2, 3, 7], q[3, 0, 1] = 1.0, INF, NAN
    wq = _rand((D,), 44, 0.1) + 1
    cache, row = mq.KV4.empty(1, 2, 2, Hkv, D, 16), torch.arange(M, dtype=torch.int32, device="cuda")
    cache.table.copy_(torch.tensor([[0, 1]]))
    out, pos, freq = torch.zeros((M, Hq, D), dtype=dtype, device="cuda"), row + 5, mq.rope_freq(n_pairs, device="cuda")
    mq.mq_qk_norm_rope_kv4(q, k, None, out, cache, None, row, pos, freq, wq=wq, wk=wq, eps=eps, interleaved=inter)
    want = _rope64(q, wq, float(torch.tensor(eps)), pos[None], freq, None, 1, inter, 1.0)
    bad = torch.isnan(want)
    assert bad[2, 3].any() and torch.equal(torch.isnan(out), bad)
    # as tests/test_gpu_kv4.py counts: 2^-20 of the pair's size for 32 bits, and the rounding to 16
    got, want = out.double().nan_to_num(0.0), want.nan_to_num(0.0)
    size_q = want.abs().amax(-1, keepdim=True) * 2 ** 0.5 + want.abs()
    assert bool(((got - want).abs() <= A.U[dtype] * want.abs() * 1.01 + 2.0 ** -20 * size_q + A.TINY[dtype]).all())
