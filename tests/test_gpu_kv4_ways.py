"""The ways that mq_attn_kv4 takes, each where the library itself takes it (seen by the workspace that it asks for): rows read into 16
bits for the tensor cores, segments finished by the blocks that hold them."""
import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as A
from tests import _kv4_ref as R
from tests._gpu_util import Guarded, require_gpu
from tests.test_gpu_kv4 import _attn_case, _inside, _rand

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture
def weights_in_f16(monkeypatch, request):
    """Weights are rounded to f16 for bf16 queries, too (the rounding that the bound counts for them otherwise is bf16's). Not for
    outputs in bf16: they are rounded by up to 2^-8 of themselves, which the bound takes from the same place."""
    if request.node.callspec.params.get("out_dtype", F32) is not BF16:
        monkeypatch.setitem(A.U, BF16, A.U[F16])
        monkeypatch.setitem(A.TINY, BF16, A.TINY[F16])


def _reads(B_, T, Hq, Hkv, D, cap):
    """Whether the workspace has room for all rows in 16 bits beside the tensor-core kernel's."""
    return mq.mq_attn_kv4_ws_bytes(B_, T, Hq, Hkv, D, cap) == 4 * B_ * cap * Hkv * D + mq.mq_attn_ws_bytes(B_, T, Hq, Hkv, D, 0, cap)


@pytest.mark.parametrize("T,Hq,Hkv,D,rows,width,lens", [(300, 28, 4, 128, 32, 64, [1900]), (320, 8, 2, 64, 64, 96, [6001, 320, 100, 0]),
                                                        (40, 32, 2, 128, 16, 400, [640, 41])])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompts_read_into_16_bits(T, Hq, Hkv, D, rows, width, lens, dtype, weights_in_f16):
    """Holes, scales that are NaN past the length, tables wider than the sequences; outputs in f32, which show the weights' type."""
    n = len(lens)
    assert _reads(n, T, Hq, Hkv, D, width * rows)
    _attn_case(T, Hq, Hkv, D, rows, lens, dtype, F32, seed=T + D, width=width, only=sorted({0, T // 2, T - 1}),
               holes=[(0, 1, -1), (0, 2, (0, 0)), (n - 1, 0, 10 ** 9)])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_in_its_own_type(dtype):
    assert _reads(1, 300, 28, 4, 128, 2048)
    _attn_case(300, 28, 4, 128, 64, [2048], dtype, seed=3, only=[0, 299])


@pytest.mark.parametrize("T,Hq,Hkv,D,lens", [(70, 8, 2, 64, [320, 100, 0, 71, 255]), (1, 8, 8, 128, [77, 1]), (3, 20, 2, 64, [200, 2, 50]),
                                             (128, 4, 1, 128, [128, 300])])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F32), (BF16, BF16), (BF16, F32)])
def test_any_rows_read_in_parts(T, Hq, Hkv, D, lens, dtype, out_dtype, weights_in_f16):
    """A test build that reads the rows of calls of any size, two sequences or so at a time."""
    own = mq.lib()
    try:
        mq._lib = mq._load(B.build_variant("kv4_read", ["MQ_KV4_READ_FROM=1", "MQ_KV4_READ_BYTES=700000"]))
        _attn_case(T, Hq, Hkv, D, 64, lens, dtype, out_dtype, seed=D + T, width=5, only=sorted({0, T // 2, T - 1}), holes=[(0, 1, -1)])
    finally:
        mq._lib = own


def _blocks_finish(n, T, Hq, Hkv, D, cap):
    """Whether the workspace is that of a call whose blocks finish the segments that they hold: 16 bytes a block behind the pieces,
    where other calls have 8 bytes a segment."""
    def up(x):
        return -(-x // 16) * 16

    rows = T * Hq // Hkv
    assert rows <= 16 and D <= 128
    nt, per_sm = (rows + 7) // 8, 12 if D == 128 and rows <= 8 or D == 96 else 16 if D == 64 and rows <= 8 else 8 if D == 128 else 12
    keys = 64 if D <= 64 or nt == 2 else 32
    segs = n * Hkv
    G = min(segs * -(-cap // keys), per_sm * torch.cuda.get_device_properties(0).multi_processor_count)
    pieces = up((G + segs) * 8 * nt * D * 4) + up((G + segs) * 8 * nt * 8)
    need = mq.mq_attn_kv4_ws_bytes(n, T, Hq, Hkv, D, cap)
    assert need in (pieces + up(16 * G), pieces + up(8 * segs))
    return segs >= G and need == pieces + up(16 * G)


@pytest.mark.parametrize("n,T,Hq,Hkv,D,rows", [(300, 1, 40, 8, 128, 64), (640, 1, 16, 4, 64, 16), (400, 3, 16, 4, 128, 32), (250, 2, 56, 8, 96, 16),
                                               (700, 2, 24, 4, 64, 64)])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, F32)])
def test_blocks_finish_their_segments(n, T, Hq, Hkv, D, rows, dtype, out_dtype, weights_in_f16):
    """Many sequences of up to 300 rows, some empty, some with fewer rows than queries, a few long ones that several blocks share; every
    seventh looked at, those and the long ones."""
    width = -(-2600 // rows)
    lens = [(37 * i) % 301 for i in range(n)]
    lens[5], lens[6], lens[n // 2], lens[-1] = 2600, 1, 2049, 1777
    assert _blocks_finish(n, T, Hq, Hkv, D, width * rows)
    pages = 300 // rows + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    P = 400
    kv = [R.round4(torch.randn((P, rows, Hkv, D), generator=g, device="cuda")) for _ in "kv"]
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    for i, m in enumerate(lens):
        used = -(-m // rows)
        table[i, :used] = torch.randint(0, P, (used,), generator=g, device="cuda").to(torch.int32)     # (sequences share pages)
    table[14, 1] = -1
    assert pages < width
    cache = mq.KV4(R.pack(*kv), table, rows, Hkv, D)
    q = _rand((n, T, Hq, D), 5, 1.5, dtype)
    out, lse = Guarded((n, T, Hq, D), out_dtype), Guarded((n, T, Hq), F32)
    mq.mq_attn_kv4(q, cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), out.t, lse=lse.t)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    out.check()
    lse.check()
    some = sorted(set(range(0, n, 49)) | {5, 6, 14, n // 2, n - 1})
    few = [lens[i] for i in some]
    k, v = R.gather(cache.pages, table[some], rows, Hkv, D, few)
    want, bound = A.attention(q[some], None, None, k, v, few, D ** -0.5, out_dtype)
    used = torch.arange(v.shape[1], device="cuda") < torch.tensor(few, device="cuda")[:, None]
    floor = 2.0 ** -32 * (v.abs() * used[..., None, None]).sum(1).repeat_interleave(Hq // Hkv, 1)[:, None]
    _inside(out.t[some], want[0], bound[0] + floor, "out")
    _inside(lse.t[some], want[1], bound[1], "lse")


def _light_key(heavy, T, dtype, cap=64, scale=0.69314718):
    """T queries whose products (base 2) are `heavy` with all keys but one, whose is less by 28; in dim 0 that key alone has a value.
    All products are whole numbers that 32 bits hold, and scale / ln 2 is 1. (output of dim 0, its value at that key, heavy keys)"""
    D, n = 64, cap - T + 1
    kn, vn = torch.zeros((1, cap, 1, D)), torch.zeros((1, cap, 1, D))
    kc, vc = torch.zeros((1, cap, 1, 2)), torch.zeros((1, cap, 1, 2))
    one, big = R.SCALES.index(1.0), R.SCALES.index(256.0)
    kn[..., 0], kc[..., 0], kc[..., 1], vc[...] = 4, big, one, one
    kn[0, 5, 0, 32], vn[0, 5, 0, 0], vn[..., 32:] = -7, 7, 3
    cache = mq.KV4(R.pack((kn, kc), (vn, vc)).cuda(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"), cap, 1, D)
    q = torch.zeros((1, T, 1, D), dtype=dtype, device="cuda")
    q[..., 0], q[..., 32] = heavy / 1024, 4.0
    assert float(torch.tensor(scale) * torch.tensor(1.4426950408889634)) == 1.0
    out = torch.full((1, T, 1, D), float("nan"), device="cuda")
    mq.mq_attn_kv4(q, cache, torch.tensor([cap], dtype=torch.int32, device="cuda"), out, scale=float(torch.tensor(scale)))
    return out[0, 0, 0, 0].item(), 7.0, n - 1


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("heavy", [2 ** 12, 2 ** 18, -2 ** 18, 2 ** 21, -2 ** 22])
def test_how_light_a_weight_may_be(heavy, T, dtype, read):
    """A weight of 2^-28 of the row's largest is there, within 2^-11 of itself and 2^-32 of the largest; where products reach 2^20
    (base 2) it may be off by 2^-25 of the largest, as include/mq.h says."""
    own = mq.lib()
    try:
        if read:
            mq._lib = mq._load(B.build_variant("kv4_read", ["MQ_KV4_READ_FROM=1", "MQ_KV4_READ_BYTES=700000"]))
        got, v, n = _light_key(heavy, T, dtype)
        torch.cuda.synchronize()
    finally:
        mq._lib = own
    p = 1.0 / (n + 2.0 ** -28)                         # of a heavy key
    floor = 2.0 ** -25 if abs(heavy) >= 2 ** 20 else 2.0 ** -32
    assert abs(got - 2.0 ** -28 * p * v) <= v * p * (max(2.0 ** -11 * 2.0 ** -28, floor) + 2.0 ** -28 * 2.0 ** -16)


@pytest.mark.parametrize("T", [1, 64])
def test_a_wide_table_and_its_first_columns(T):
    """640 rows in a table for 131072: right as it is, and the same bits and workspace as a table for 640 where only its first columns are
    given."""
    n, Hq, Hkv, D, rows, width = 2, 40, 8, 128, 64, 2048
    cache = R.random_cache(n, 10, rows, Hkv, D, 61)
    wide = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    wide[:, :10] = cache.table
    lens = [640, 577]
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = _rand((n, T, Hq, D), 62, 1.0, F16)
    out = []
    for table in (cache.table, wide[:, :10], wide):
        c = mq.KV4(cache.pages, table, rows, Hkv, D)
        out.append(torch.full((n, T, Hq, D), float("nan"), device="cuda"))
        mq.mq_attn_kv4(q, c, length, out[-1], ws=mq.attn_kv4_workspace(n, T, Hq, Hkv, D, c.cap))
    assert torch.equal(out[0], out[1])
    assert mq.mq_attn_kv4_ws_bytes(n, T, Hq, Hkv, D, 640) < mq.mq_attn_kv4_ws_bytes(n, T, Hq, Hkv, D, width * rows)
    k, v = R.gather(cache.pages, cache.table, rows, Hkv, D, lens)
    some = sorted({0, T - 1})
    want, bound = A.attention(q, None, None, k, v, lens, D ** -0.5, F32, only=some)
    for o in out:
        _inside(o[:, some], want[0][:, some], bound[0][:, some] + 2.0 ** -32 * v.abs().sum(), "out")
