"""The calls on 4-bit caches against plain forms in 64 bits: what is written byte for byte, rows read back exactly,
attention within the bound of its arithmetic (tests/_attn_ref.py: keys and values are exact in 16 bits, so it is
mq_attn_prefix's)."""
import math

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as A
from tests import _kv4_ref as R
from tests._gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rand(shape, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _rope64(x, w, eps, pos, freq, axis, n_axes, interleaved, turn):
    """Norm and rotation in 64 bits, [M, H, D]."""
    y = x.double()
    if w is not None:
        y = y * w.double() / ((y * y).mean(-1, keepdim=True) + eps).sqrt()
    n = 0 if freq is None else freq.numel()
    out = y.clone()
    for i in range(n):
        ax = 0 if axis is None else min(int(axis[i]), n_axes - 1)
        t = pos[ax].double() * freq[i].double()
        c, s = (t.cos() * turn)[:, None], (t.sin() * turn)[:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., ia], out[..., ib] = y[..., ia] * c - y[..., ib] * s, y[..., ia] * s + y[..., ib] * c
    return out


def _fill_case(M, Hq, Hkv, D, page_rows, n, n_pairs, dtype=F16, norm=True, inter=False, axes=1, turn=1.0, seed=0, std=1.0,
               x=None, holes=False):
    q = _rand((M, Hq, D), seed, std)
    kv = _rand((M, 2 * Hkv, D), seed + 1, std) if x is None else x
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    wq, wk = ((_rand((D,), seed + 2 + i, 0.1) + 1) if norm else None for i in range(2))
    freq = mq.rope_freq(n_pairs, device="cuda") if n_pairs else None
    g = torch.Generator()
    g.manual_seed(seed)
    pos = torch.randint(-5, 200000, (axes, M), generator=g).to(torch.int32).cuda()
    axis = (torch.arange(n_pairs, dtype=torch.uint8) % 4).cuda() if axes > 1 else None
    width = max(1, -(-2 * M // (n * page_rows)))
    P = n * width + 2
    place = torch.randperm(n * width * page_rows, generator=g)[:M]
    seq, row = (place // (width * page_rows)).to(torch.int32), (place % (width * page_rows)).to(torch.int32)
    if M > 3:
        seq[0], row[1], row[2] = n, -1, width * page_rows         # nowhere
    table = torch.randperm(P, generator=g)[:n * width].to(torch.int32).view(n, width)
    if holes:
        table[0, 0] = -1
        table[-1, -1] = P
    size = mq.mq_kv4_page_bytes(page_rows, Hkv, D)
    pages = Guarded((P, size), torch.uint8)
    cache = mq.KV4(pages.t, table.cuda(), page_rows, Hkv, D)
    q_out = Guarded((M, Hq, D), dtype)
    turn = float(torch.tensor(turn))
    mq.mq_qk_norm_rope_kv4(q, k, v, q_out.t, cache, seq.cuda(), row.cuda(), pos, freq, axis=axis, wq=wq, wk=wk, eps=1e-6,
                           interleaved=inter, rot_scale=turn)
    torch.cuda.synchronize()
    pages.check()
    q_out.check()
    eps = float(torch.tensor(1e-6))
    want_q = _rope64(q, wq, eps, pos, freq, axis, axes, inter, turn)
    # the roundings that tests/_attn_ref.py counts for rope(), with those of rot_scale in the same 2^-20 of the pair's size
    size_q = want_q.abs().amax(-1, keepdim=True) * math.sqrt(2) + want_q.abs()
    # (past the type's largest number an infinity is the rounding)
    over = torch.isinf(want_q.to(dtype))
    assert torch.equal(q_out.t[over], want_q.to(dtype)[over])
    want_q, got_q = want_q.masked_fill(over, 0.0), q_out.t.double().masked_fill(over, 0.0)
    assert bool(((got_q - want_q).abs() <= A.U[dtype] * want_q.abs() * 1.01 + 2.0 ** -20 * size_q + A.TINY[dtype]).all())
    kn, vn = R.round4(_rope64(k, wk, eps, pos, freq, axis, axes, inter, turn)), R.round4(v)
    # every byte: those of rows that were written, and nothing else (poison 0xCD)
    kb, ks, vb, vs, kc, vc = (t.cuda() for t in R.places(D))
    want = torch.full((P, Hkv, page_rows // 16, R.block_bytes(D)), 0xCD, dtype=torch.long, device="cuda")
    tbl = table.tolist()
    for m in range(M):
        s, r = int(seq[m]), int(row[m])
        if not (0 <= s < n and 0 <= r < width * page_rows) or not 0 <= tbl[s][r // page_rows] < P:
            continue
        page, blk, i = tbl[s][r // page_rows], r % page_rows // 16, r % 16
        for (num, code), at, shift, cat in ((kn, kb, ks, kc), (vn, vb, vs, vc)):
            b = want[page, :, blk]
            nib = num[m].long() + 8
            for sh in (0, 4):
                sel = shift[i] == sh
                old = b[:, at[i][sel]]
                b[:, at[i][sel]] = (old & (0xF0 if sh == 0 else 0x0F)) | (nib[:, sel] << sh)
            b[:, cat[i]] = code[m]
    got = cache.pages.view(P, Hkv, page_rows // 16, R.block_bytes(D)).long()
    bad = (got != want).nonzero()
    assert len(bad) == 0, f"{len(bad)} bytes differ, first {bad[:4].tolist()}"


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_fill_widths(D, inter):
    _fill_case(37, 6, 2, D, 32, 2, D // 2, inter=inter, seed=D)


@pytest.mark.parametrize("M,Hq,Hkv,page_rows,n", [(1, 40, 8, 64, 1), (2, 3, 3, 16, 1), (50, 28, 4, 16, 3), (333, 12, 1, 256, 2),
                                                  (700, 4, 4, 1024, 1)])
def test_fill_sizes(M, Hq, Hkv, page_rows, n):
    _fill_case(M, Hq, Hkv, 128, page_rows, n, 64, dtype=BF16, seed=M, holes=M > 40)


@pytest.mark.parametrize("n_pairs,inter", [(0, False), (1, False), (30, False), (30, True), (48, False), (60, False), (61, True)])
@pytest.mark.parametrize("norm", [False, True])
def test_fill_partial_rotation(n_pairs, inter, norm):
    _fill_case(40, 2, 3, 128, 64, 2, n_pairs, norm=norm, inter=inter, seed=n_pairs)


def test_fill_axes_and_scaled():
    _fill_case(100, 4, 2, 128, 64, 1, 64, axes=3, turn=1.2772588722, seed=5)
    _fill_case(100, 4, 2, 64, 64, 1, 32, turn=-0.3, seed=6)


@pytest.mark.parametrize("std", [1e-6, 3e-4, 30.0, 2e3, 1e6])
def test_fill_scales(std):
    """Below the least scale, in the subnormal ones, and past the largest."""
    _fill_case(64, 2, 2, 128, 64, 1, 64, norm=False, seed=9, std=std)


def test_fill_norm_of_any_size():
    """Heads whose mean square 32 bits do not hold, and zeros, normed."""
    M, H, D = 24, 2, 64
    x = _rand((M, H, D), 91)
    x *= (10.0 ** torch.linspace(-30, 30, M, device="cuda"))[:, None, None]
    x[5, 0] = 0.0
    cache = mq.KV4.empty(1, 2, 2, H, D, 16)
    cache.table.copy_(torch.tensor([[1, 0]]))
    cache.pages.zero_()
    wk, row = _rand((D,), 92, 0.1) + 1, torch.arange(M, dtype=torch.int32, device="cuda")
    freq, pos = mq.rope_freq(32, device="cuda"), row + 3
    for eps in (1e-6, 0.0):
        mq.mq_qk_norm_rope_kv4(None, x, None, None, cache, None, row, pos, freq, wk=wk, eps=eps)
        y = _rope64(x, wk, float(torch.tensor(eps)), pos[None], freq, None, 1, False, 1.0)
        want = R.value4(*R.round4(y))
        got = R.unpack(cache.pages[[1, 0]], 16, H, D)[0].flatten(0, 1)[:M]
        bad = ((got != want) & torch.isfinite(y)).nonzero()          # (zeros over zero have no value)
        assert len(bad) == 0, (eps, len(bad), bad[:4].tolist(), [(float(y[tuple(b)]), float(got[tuple(b)])) for b in bad[:4].tolist()])


def test_fill_ties_and_grid():
    """Rows whose numbers lie on borders, whose largest lies on a scale's, and zeros."""
    M, H, D = 96, 2, 128
    x = torch.zeros((M, 2 * H, D), device="cuda")
    for m in range(M):
        c = 8 + 2 * m - (m == 95)
        d = R.SCALES[min(c, R.MOST)]
        i = torch.arange(D, device="cuda")
        x[m] = (((i * 7 + m) % 29) - 14) * 0.5 * d          # multiples of d / 2 up to 7 d
        x[m, 1, :32] = 0.0
        x[m, 2] *= 1 + 2.0 ** -23                          # next to the border
        x[m, 3] *= 1 - 2.0 ** -24
    x[0, 0], x[1, 2] = 0.0, -0.0
    _fill_case(M, 2, H, D, 32, 1, 0, norm=False, x=x)


def test_fill_many_rows():
    """Enough rows that some lie next to a border for 32 bits: 4096 x 8 heads."""
    M, H, D, rows = 4096, 8, 128, 128
    k, v = _rand((M, H, D), 1), _rand((M, H, D), 2)
    wk = _rand((D,), 3, 0.1) + 1
    freq, pos = mq.rope_freq(64, device="cuda"), torch.arange(M, dtype=torch.int32, device="cuda") + 77777
    cache = mq.KV4.empty(1, M // rows, M // rows, H, D, rows)
    cache.table.copy_(torch.arange(M // rows, device="cuda").view(1, -1))
    mq.mq_qk_norm_rope_kv4(None, k, v, None, cache, None, torch.arange(M, dtype=torch.int32, device="cuda"), pos, freq, wk=wk)
    eps = float(torch.tensor(1e-6))
    want = R.pack(*(tuple(t.view(M // rows, rows, H, -1) for t in R.round4(x))
                    for x in (_rope64(k, wk, eps, pos[None], freq, None, 1, False, 1.0), v)))
    assert torch.equal(cache.pages, want)


def test_fill_leaves_out():
    """Only keys, only values, only queries."""
    M, H, D, rows = 20, 2, 64, 16
    k, v, q = (_rand((M, H, D), i) for i in range(3))
    row = torch.arange(M, dtype=torch.int32, device="cuda")
    want = R.pack(*(tuple(torch.cat([t, torch.zeros_like(t[:12])]).view(2, rows, H, -1) for t in R.round4(x)) for x in (k, v)))
    nothing = R.pack(*(tuple(torch.zeros((2, rows, H, n), device="cuda") - (8 if n == D else 0) for n in (D, D // 32)) for _ in "kv"))
    keys = torch.zeros_like(want[0], dtype=torch.bool).view(H, 1, -1)
    keys[..., :8 * D] = keys[..., 16 * D:16 * D + D // 2] = True
    for a, b in ((k, None), (None, v), (None, None)):
        cache = mq.KV4.empty(1, 2, 2, H, D, rows)
        cache.table.copy_(torch.tensor([[0, 1]]))
        cache.pages.zero_()
        out = torch.empty((M, H, D), dtype=F16, device="cuda")
        mq.mq_qk_norm_rope_kv4(q, a, b, out, cache, None, row)
        assert torch.equal(out, q.half())
        sel = keys.flatten() if a is not None else ~keys.flatten() if b is not None else torch.zeros_like(keys.flatten())
        got = cache.pages.clone()
        assert not got[:, ~sel].any()
        # rows 20 .. 31 stay zero bytes where the wanted ones have nibbles of 8
        mask = got != 0
        assert torch.equal(got[mask], torch.where(sel, want, torch.zeros_like(want))[mask])
        if a is not None or b is not None:
            ku, vu = R.unpack(got, rows, H, D)
            x, u = (k, ku) if a is not None else (v, vu)
            assert torch.equal(u.flatten(0, 1)[:M], R.value4(*R.round4(x)))
    del nothing


# ------------------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_read(D, dtype):
    n, width, rows, H = 3, 3, 32, 3
    cache = R.random_cache(n, width, rows, H, D, D)
    cache.table[1, 1], cache.table[2, 0] = -1, 10 ** 6
    length = torch.tensor([70, 96, 41], dtype=torch.int32, device="cuda")
    k, v = (Guarded((n, 90, H, D), dtype) for _ in range(2))
    poison = k.t.clone()
    mq.mq_kv4_read(cache, length, mq.KV(k.t, v.t))
    torch.cuda.synchronize()
    want = R.gather(cache.pages, cache.table, rows, H, D, [70, 90, 41])
    for got, w in zip((k, v), want):
        got.check()
        for i, m in enumerate((70, 90, 41)):
            assert torch.equal(got.t[i, :m].double(), w[i, :m])
            assert torch.equal(got.t[i, m:].view(torch.int16), poison[i, m:].view(torch.int16))


def test_read_every_scale():
    """All scale bytes up to the largest, all numbers -8 .. 7, exactly, in both types."""
    H, D, rows = 1, 128, 64
    code = torch.arange(192).repeat_interleave(2)[:, None, None].expand(-1, 1, 4).contiguous().view(6, rows, H, 4)
    num = ((torch.arange(384 * D) * 5 + torch.arange(384 * D) // 16) % 16 - 8).view(6, rows, H, D)
    pages = R.pack((num, code), (num.flip(-1), code)).cuda()
    cache = mq.KV4(pages, torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6), rows, H, D)
    for dtype in (F16, BF16):
        kv = mq.KV.empty(1, 384, H, D, dtype)
        mq.mq_kv4_read(cache, torch.tensor([384], dtype=torch.int32, device="cuda"), kv)
        for got, x in ((kv.k, num), (kv.v, num.flip(-1))):
            want = R.value4(x, code).flatten(0, 1).cuda()
            assert torch.equal(got[0].double(), want)


def test_read_strides():
    n, width, rows, H, D = 2, 2, 16, 4, 64
    cache = R.random_cache(n, width, rows, H, D, 3)
    wide = torch.zeros((2, 6), dtype=torch.int32, device="cuda")
    wide[:, 1:3] = cache.table
    big = torch.zeros((cache.n_pages, cache.pages.shape[1] + 48), dtype=torch.uint8, device="cuda")
    big[:, :cache.pages.shape[1]] = cache.pages
    with pytest.raises(mq.MQError):                    # a table that does not begin on 16 bytes
        mq.mq_kv4_read(mq.KV4(big, wide[:, 1:3], rows, H, D), torch.zeros(2, dtype=torch.int32, device="cuda"), mq.KV.empty(n, 32, H, D))
    wide[:, :2] = cache.table
    strided = mq.KV4(big, wide[:, :2], rows, H, D)
    length = torch.tensor([32, 17], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((n, H, 40, D), dtype=F16, device="cuda") for _ in range(2))
    mq.mq_kv4_read(strided, length, mq.KV(k.transpose(1, 2), v.transpose(1, 2)))
    want = R.gather(cache.pages, cache.table, rows, H, D, [32, 17])
    for got, w in zip((k, v), want):
        for i, m in enumerate((32, 17)):
            assert torch.equal(got[i, :, :m].transpose(0, 1).double(), w[i, :m])
            assert not got[i, :, m:].any()


# ------------------------------------------------------------------------------------------- attention

@pytest.fixture(params=["as it is", "finished by blocks"])
def finish(request):
    """The library, and a test build that finishes segments in the blocks that hold them in calls of any size (the library: from
    609 query rows on)."""
    own = mq.lib()
    if request.param != "as it is":
        mq._lib = mq._load(B.build_variant("kv4_split", ["MQ_KV4_SPLIT_FROM=0", "MQ_TEST_INJECT", "MQ_WAIT_LIMIT_NS=50000000ull"]))
    yield
    mq._lib = own


def _inside(got, want, bound, what):
    got = got.double()
    assert not torch.isnan(got).any(), f"{what}: NaN"
    same = got == want
    bad = ~same & ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst error / bound " \
        f"{float(((got - want).abs() / bound)[~same].max()):.3g}"


def _attn_case(T, Hq, Hkv, D, rows, lens, dtype=F16, out_dtype=None, seed=0, std=1.5, width=None, holes=(), scale=None, only=None,
               k_std=1.0):
    n = len(lens)
    width = width or max(1, -(-max(max(lens), 1) // rows))
    cache = R.random_cache(n, width, rows, Hkv, D, seed, std=k_std)
    for i, j, p in holes:
        cache.table[i, j] = cache.table[p] if isinstance(p, tuple) else p
    k, v = R.gather(cache.pages, cache.table, rows, Hkv, D, lens)
    # what lies past a sequence's length must not matter, whatever it is
    for i, m in enumerate(lens):
        m = max(0, min(m, width * rows))
        if m % 16 and 0 <= int(cache.table[i, m // rows]) < cache.n_pages:
            p, blk = int(cache.table[i, m // rows]), m % rows // 16
            _, _, vb, vs, kc, vc = R.places(D)
            b = cache.pages[p].view(Hkv, rows // 16, R.block_bytes(D))
            for r in range(m % 16, 16):
                b[:, blk, kc[r].cuda()] = 255
                b[:, blk, vc[r].cuda()] = 255
    q = _rand((n, T, Hq, D), seed + 5, std, dtype)
    out_dtype = out_dtype or dtype
    out, lse = Guarded((n, T, Hq, D), out_dtype), Guarded((n, T, Hq), F32)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = D ** -0.5 if scale is None else scale
    mq.mq_attn_kv4(q, cache, length, out.t, scale=scale, lse=lse.t)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    want, bound = A.attention(q, None, None, k, v, lens, scale, out_dtype, only=only)
    # Weights are in f16 for bf16 queries too: the largest of a row is 2^7 or more, half of f16's least step 2^-25, and the sum
    # no less than the largest, so besides 2^-8 (2^-11) of itself a weight is off by at most 2^-32. Seen where the values of all
    # heavier keys are zeros.
    used = torch.arange(v.shape[1], device="cuda") < length[:, None]
    floor = 2.0 ** -32 * (v.abs() * used[..., None, None]).sum(1).repeat_interleave(Hq // Hkv, 1)[:, None]
    bound = (bound[0] + floor, bound[1])
    sel = slice(None) if only is None else only
    _inside(out.t[:, sel], want[0][:, sel], bound[0][:, sel], "out")
    _inside(lse.t[:, sel], want[1][:, sel], bound[1][:, sel], "lse")
    out.check()
    lse.check()
    assert out.untouched() == 0 or out_dtype == F16 and out.untouched() < 4
    return cache, q, length, out.t, lse.t


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 3])
def test_attention_widths(D, dtype, T, finish):
    _attn_case(T, 8, 2, D, 32, [1, 16, 31, 33, 64, 100, 0, 150], dtype, seed=D + T)


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 1024])
def test_attention_pages(rows, finish):
    _attn_case(1, 7, 1, 128, rows, [5, 15, 17, 200, 129, 1000], BF16, seed=rows)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (9, 1), (17, 1), (25, 1), (33, 1), (28, 4), (64, 8), (70, 2)])
def test_attention_groups(Hq, Hkv, finish):
    _attn_case(1, Hq, Hkv, 128, 64, [77, 1, 300], F16, seed=Hq)


@pytest.mark.parametrize("T", [2, 5, 8, 16, 19])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_several_queries(T, D, finish):
    """Fewer rows than queries, too: those queries see nothing."""
    _attn_case(T, 12, 3, D, 16, [T, T + 1, 40, 97, 1, 0, T - 1], BF16, seed=T)


@pytest.mark.parametrize("out_dtype", [F16, BF16, F32])
def test_attention_out_types(out_dtype, finish):
    _attn_case(1, 8, 2, 128, 64, [100, 31], BF16 if out_dtype == BF16 else F16, out_dtype, seed=1)


def test_attention_long(finish):
    """Several blocks a sequence, ragged, with pieces joined."""
    _attn_case(1, 40, 8, 128, 64, [9000, 17, 20011, 1], F16, seed=2)
    _attn_case(4, 14, 2, 64, 32, [5000, 3, 12345], BF16, seed=3)


def test_attention_light_weights(finish):
    """Dims whose value is zero at all keys but the lightest, in full precision."""
    _attn_case(1, 36, 3, 256, 1024, [3, 0, 1, 6, 6, 4, 1], BF16, out_dtype=F32, seed=267439, std=6.0)


def test_attention_many_sequences():
    """Enough rows that the library itself finishes segments in their blocks; some sequences are empty."""
    lens = [(37 * i) % 150 for i in range(90)] + [0, 1, 2500]
    _attn_case(1, 8, 2, 128, 32, lens, F16, seed=77)
    _attn_case(2, 8, 2, 64, 16, lens[:60], BF16, F32, seed=78)


def test_attention_holes(finish):
    """Entries that are no page read as zero rows."""
    _attn_case(1, 8, 2, 128, 16, [100, 64, 16], F16, seed=4, holes=[(0, 1, -1), (0, 4, 10 ** 9), (1, 3, (0, 2)), (2, 0, -7)])
    _attn_case(2, 8, 2, 64, 64, [200, 64], BF16, seed=5, holes=[(0, 1, -1), (1, 0, -2 ** 31)])
    _attn_case(60, 8, 2, 128, 64, [200, 130], F16, seed=6, holes=[(0, 1, -1), (1, 0, 5000)], only=[0, 31, 59])


def test_attention_lengths_outside(finish):
    """Negative lengths are empty, those past the table end at it."""
    cache, q, _, _, _ = _attn_case(1, 4, 2, 64, 16, [32, 48], F16, seed=7, width=3)
    out = torch.empty_like(q)
    mq.mq_attn_kv4(q, cache, torch.tensor([-5, 10 ** 9], dtype=torch.int32, device="cuda"), out)
    want = torch.empty_like(q)
    mq.mq_attn_kv4(q, cache, torch.tensor([0, 48], dtype=torch.int32, device="cuda"), want)
    assert not out[0].any() and torch.equal(out, want)


@pytest.mark.parametrize("T,Hq,Hkv,D,lens", [(64, 8, 2, 128, [64, 200, 30]), (130, 7, 1, 64, [130, 512]), (33, 16, 4, 96, [90, 33]),
                                             (40, 8, 4, 256, [111, 40]), (300, 28, 4, 128, [1300])])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_prompts(T, Hq, Hkv, D, lens, dtype):
    _attn_case(T, Hq, Hkv, D, 32, lens, dtype, seed=T, only=sorted({0, 1, T // 2, T - 1}))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-3, 3.0])
def test_attention_scales(scale):
    _attn_case(1, 4, 1, 128, 32, [70, 9], F16, seed=8, scale=scale)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_large_products(dtype, finish):
    """Products of 2^20 and more, with the maximum growing from tile to tile."""
    _attn_case(1, 4, 1, 64, 32, [200], dtype, seed=9, std=300.0, k_std=60.0, scale=3.0)


def test_attention_strided_queries_and_stream():
    n, Hq, Hkv, D = 3, 8, 2, 128
    cache = R.random_cache(n, 4, 32, Hkv, D, 11)
    length = torch.tensor([100, 128, 7], dtype=torch.int32, device="cuda")
    wide = _rand((n, 1, Hq + 4, D), 12, 1.0, F16)
    q = wide[:, :, 2:2 + Hq]
    want, out = (torch.zeros((n, 1, Hq, D), dtype=F16, device="cuda") for _ in range(2))
    mq.mq_attn_kv4(q.contiguous(), cache, length, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mq.mq_attn_kv4(q, cache, length, out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_attention_row_is_its_own(finish):
    """A row's bits do not depend on its neighbours' numbers."""
    n, Hq, Hkv, D = 2, 16, 2, 128
    cache = R.random_cache(n, 8, 64, Hkv, D, 13)
    length = torch.tensor([500, 333], dtype=torch.int32, device="cuda")
    q = _rand((n, 1, Hq, D), 14, 1.0, F16)
    a, b = (torch.zeros((n, 1, Hq, D), dtype=F16, device="cuda") for _ in range(2))
    mq.mq_attn_kv4(q, cache, length, a)
    other = q.clone()
    other[:, :, 1::2] = _rand((n, 1, Hq // 2, D), 15, 20.0, F16)
    other[0, 0, 3] = float("nan")
    mq.mq_attn_kv4(other, cache, length, b)
    assert torch.equal(a[:, :, ::2], b[:, :, ::2]) and torch.isnan(b[0, 0, 3]).all()


def test_calls_in_a_graph():
    """Fill, read and attention captured once, replayed with other lengths, tables and inputs."""
    n, Hq, Hkv, D, rows, width = 2, 8, 2, 128, 16, 6
    cache = R.random_cache(n, width, rows, Hkv, D, 21)
    q, k, v = (_rand((n, h, D), 22 + h) for h in (Hq, Hkv, Hkv + 1))
    v = v[:, :Hkv].contiguous()
    seq, row = torch.arange(n, dtype=torch.int32, device="cuda"), torch.tensor([3, 40], dtype=torch.int32, device="cuda")
    length, pos, freq = row + 1, row + 9, mq.rope_freq(64, device="cuda")
    q16, out = torch.zeros((n, Hq, D), dtype=F16, device="cuda"), torch.zeros((n, 1, Hq, D), dtype=F16, device="cuda")
    kv = mq.KV.empty(n, width * rows, Hkv, D)
    ws = mq.attn_kv4_workspace(n, 1, Hq, Hkv, D, cache.cap)

    def step():
        mq.mq_qk_norm_rope_kv4(q, k, v, q16, cache, seq, row, pos, freq)
        mq.mq_attn_kv4(q16.view(n, 1, Hq, D), cache, length, out, ws=ws)
        mq.mq_kv4_read(cache, length, kv)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        row.copy_(torch.tensor([5 + 20 * i, 41 + i]))
        length.copy_(row + 1)
        pos.copy_(row + 2)
        q.copy_(_rand(q.shape, 30 + i))
        cache.table.copy_(cache.table.flip(1))
        keep = cache.pages.clone()
        graph.replay()
        torch.cuda.synchronize()
        got, pages = (out.clone(), kv.k.clone()), cache.pages.clone()
        cache.pages.copy_(keep)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(pages, cache.pages)
        for b in range(n):
            assert torch.equal(got[1][b, :int(length[b])], kv.k[b, :int(length[b])])


def test_offsets_past_2_31():
    """Pages more than 2^32 bytes from the pool's start, and tokens' rows there."""
    H, D, rows = 8, 128, 1024
    size = mq.mq_kv4_page_bytes(rows, H, D)
    P = (1 << 32) // size + 5
    pages = torch.empty((P, size), dtype=torch.uint8, device="cuda")
    small = R.random_cache(1, 2, rows, H, D, 41, spare=0)
    pages[P - 2:] = small.pages
    far = mq.KV4(pages, (small.table + P - 2).contiguous(), rows, H, D)
    q = _rand((1, 1, 16, D), 42, 1.0, BF16)
    length = torch.tensor([1900], dtype=torch.int32, device="cuda")
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    mq.mq_attn_kv4(q, small, length, a)
    mq.mq_attn_kv4(q, far, length, b)
    assert torch.equal(a, b) and a.any()
    k, v = _rand((5, H, D), 43), _rand((5, H, D), 44)
    row = torch.tensor([1900, 1901, 1902, 2047, 0], dtype=torch.int32, device="cuda")
    for c in (small, far):
        mq.mq_qk_norm_rope_kv4(None, k, v, None, c, None, row)
    assert torch.equal(pages[P - 2:], small.pages)


@pytest.mark.parametrize("n", [2, 5])
def test_prompt_read_into_16_bits(n):
    """A test build that reads the rows of calls of any size into 16 bits, those of two sequences at a time."""
    T, Hq, Hkv, D = 70, 8, 2, 128
    cache = R.random_cache(n, 5, 64, Hkv, D, 51)
    lens = [320, 100, 0, 71, 255][:n]
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = _rand((n, T, Hq, D), 52, 1.0, F16)
    own = mq.lib()
    try:
        mq._lib = mq._load(B.build_variant("kv4_read", ["MQ_KV4_READ_FROM=1", "MQ_KV4_READ_BYTES=700000"]))
        out, lse = torch.zeros_like(q), torch.zeros((n, T, Hq), device="cuda")
        mq.mq_attn_kv4(q, cache, length, out, lse=lse)
        torch.cuda.synchronize()
        assert mq.mq_device_status() == mq.MQ_OK
    finally:
        mq._lib = own
    k, v = R.gather(cache.pages, cache.table, 64, Hkv, D, lens)
    some = [0, 35, 69]
    want, bound = A.attention(q, None, None, k, v, lens, D ** -0.5, F16, only=some)
    _inside(out[:, some], want[0][:, some], bound[0][:, some], "out")
    _inside(lse[:, some], want[1][:, some], bound[1][:, some], "lse")
