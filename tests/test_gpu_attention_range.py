"""mq_attn_prefix where the exponents' range and rounding matter: products far past what 16 bits hold, many small weights
beside a dominant one, scales of next to nothing. Every test runs on the library as it is and on a test build that sends calls of
any size to the tensor-core kernel."""
import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import require_gpu

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


@pytest.mark.parametrize("dtype,std", [(F16, 300.0), (F16, 3000.0), (F16, 12000.0), (BF16, 1e6), (BF16, 1e10), (BF16, 1e15)])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_products_of_any_size_pick_a_key(T, dtype, std):
    """Finite operands whose products are far apart: one key has all the weight, and the output is its value. A query
    counts if its two best keys are 200 apart beyond what f32 sums of the products can be off by (2^-16 of the sum of their
    sizes); the output is then off by one rounding of the weight and one of its own, and by 2^-18 for the exponential."""
    Hq, Hkv, D, P, cap = 4, 2, 128, 200, T + 400
    q = _rand((1, T, Hq, D), dtype, T, std).clamp(-5 * std, 5 * std)
    pk, k = (_rand((1, n, Hkv, D), dtype, T + i, std).clamp(-5 * std, 5 * std) for i, n in ((1, P), (2, cap)))
    pv, v = _rand((1, P, Hkv, D), dtype, T + 3), _rand((1, cap, Hkv, D), dtype, T + 4)
    n = torch.tensor([cap - 3], dtype=torch.int32, device="cuda")
    out, lse = torch.empty((1, T, Hq, D), device="cuda"), torch.empty((1, T, Hq), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), n, out, lse=lse)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    counted = 0
    for h in range(Hq):
        K = torch.cat([pk[0, :, h // 2], k[0, :, h // 2]]).double()
        V = torch.cat([pv[0, :, h // 2], v[0, :, h // 2]]).double()
        x = q[0, :, h].double()
        s = x @ K.T * D ** -0.5
        size = x.abs() @ K.abs().T * D ** -0.5
        late = torch.arange(P + cap, device="cuda") >= (P + cap - 3 - T + 1 + torch.arange(T, device="cuda"))[:, None]
        s.masked_fill_(late, -float("inf"))
        top = s.topk(2, dim=-1)
        off = 2.0 ** -16 * size.masked_fill(late, 0.0).amax(-1)
        clear = top.values[:, 0] - top.values[:, 1] > 200 + 2 * off
        counted += int(clear.sum())
        want = V[top.indices[:, 0]]
        bad = ~((out[0, :, h].double() - want).abs() <= want.abs() * (R.U[dtype] + 2.0 ** -18))
        assert not bad[clear].any(), f"head {h}: {int(bad[clear].sum())} values of other keys, or none"
        assert bool(((lse[0, :, h].double() - top.values[:, 0]).abs() <= off + 1e-3)[clear].all())
    assert counted > (0.9 if std > 1000 else 0.5) * T * Hq


def test_a_later_tile_just_above_the_maximum():
    """Two products of 2^20 and 2^20 + 1/8 times a scale around 100: the scaled ones are 16 apart, one unit in the last
    place, in different key tiles. Whatever weights that gives, the outputs lie between the two values."""
    D, cap = 64, 300
    q = torch.zeros((1, 30, 1, D), dtype=F16, device="cuda")
    q[..., 0], q[..., 1] = 1024.0, 0.125
    k = torch.zeros((1, cap, 1, D), dtype=F16, device="cuda")
    k[..., 0] = 1024.0
    k[:, 200:, :, 1] = 1.0
    v = torch.ones((1, cap, 1, D), dtype=F16, device="cuda")
    v[:, 200:] = 2.0
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    for i in range(60):
        out = torch.empty((1, 30, 1, D), device="cuda")
        mq.mq_attn_prefix(q, None, mq.KV(k, v), n, out, scale=91.0 + 1.37 * i)
        assert bool(((out >= 1 - 2.0 ** -10) & (out <= 2 + 2.0 ** -9)).all()), i


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,P,cap", [(1, 0, 16), (1, 0, 700), (1, 40000, 10), (3, 33000, 200), (20, 5000, 300), (600, 40000, 1000),
                                     (700, 0, 700)])
def test_many_small_weights_beside_a_dominant_one(T, P, cap, dtype):
    """The first key outweighs each of the others some 2^25.5 times, and its value is zero: the output is what the others
    add up to, and none may be lost for being small beside the first. Off by a rounding of each weight (relative, or half of
    f16's smallest number against a weight of 2^7 for the maximum), by 2^-15 for the exponentials of products up to 18, by 2^-16 for
    the sums."""
    D, Hq = 64, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(P + cap)
    q = torch.zeros((1, T, Hq, D), dtype=dtype, device="cuda")
    q[..., 0] = 8.0                                        # times a scale of 1/8: products are the keys' first element
    N = P + cap
    keys, vals = (torch.zeros((N, 1, D), dtype=dtype, device="cuda") for _ in range(2))
    keys[1:, 0, 0] = (-17.675 + 0.3 * torch.randn(N - 1, generator=g, device="cuda").clamp(-2, 2)).to(dtype)
    vals[1:, 0] = (0.5 + 0.5 * torch.rand((N - 1, D), generator=g, device="cuda")).to(dtype)
    pre = mq.KV(keys[None, :P], vals[None, :P]) if P else None
    out = torch.empty((1, T, Hq, D), device="cuda")
    mq.mq_attn_prefix(q, pre, mq.KV(keys[None, P:], vals[None, P:]), torch.full((1,), cap, dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    p = keys[:, 0, 0].double().exp()
    sees = (N - T + 1 + torch.arange(T, device="cuda")) - 1                       # last key that each query sees
    total = p.cumsum(0)[sees][:, None]
    want = (p[:, None] * vals[:, 0].double()).cumsum(0)[sees] / total
    mass = vals[:, 0].double().cumsum(0)[sees] / total
    bound = want * (R.U[dtype] + 2.0 ** -15 + 2.0 ** -16) + (2.0 ** -32 * mass if dtype is F16 else 0.0) + 2.0 ** -24 * want
    bad = (out[0].double() - want[:, None]).abs() > bound[:, None]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; worst relative error " \
        f"{float(((out[0].double() - want[:, None]).abs() / want[:, None]).max()):.3g}"


@pytest.mark.parametrize("scale", [0.0, 1e-38, 3e-33, -3e-33])
@pytest.mark.parametrize("T", [1, 50])
def test_scales_of_next_to_nothing(T, scale):
    """Products of some 1e32: a scale of zero weighs all keys alike, one of 3e-33 does not quite."""
    B, Hq, Hkv, D, P, cap = 2, 4, 2, 64, 70, 200
    q, k, v = (_rand((B, n, h, D), BF16, i, s) for i, (n, h, s) in enumerate(((T, Hq, 3e15), (cap, Hkv, 3e15), (cap, Hkv, 1.0))))
    pk, pv = _rand((1, P, Hkv, D), BF16, 5, 3e15), _rand((1, P, Hkv, D), BF16, 6)
    lens = [cap, T + 20]
    out, lse = torch.empty((B, T, Hq, D), device="cuda"), torch.empty((B, T, Hq), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, scale=scale, lse=lse)
    want, bound = R.attention(q, pk[0], pv[0], k, v, lens, scale, F32)
    assert bool(((out.double() - want[0]).abs() <= bound[0]).all())
    assert bool(((lse.double() - want[1]).abs() <= bound[1]).all())


@pytest.mark.parametrize("T", [1, 3])
def test_more_sequences_and_heads_than_a_grid_axis(T):
    """8200 sequences of 8 key heads, most of them short; sampled ones against the reference."""
    B, H, D, P, cap = 8200, 8, 64, 20, 6
    q, k, v = (_rand((B, n, H, D), F16, i) for i, n in enumerate((T, cap, cap)))
    pk, pv = _rand((1, P, H, D), F16, 3), _rand((1, P, H, D), F16, 4)
    lens = [(5 * b) % (cap + 1) for b in range(B)]
    out = torch.empty((B, T, H, D), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv), mq.KV(k, v), torch.tensor(lens, dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    for b in (0, 1, 4099, 8190, 8191, 8192, 8199):
        want, bound = R.attention(q[b:b + 1], pk[0], pv[0], k[b:b + 1], v[b:b + 1], lens[b:b + 1], D ** -0.5, F32)
        assert bool(((out[b:b + 1].double() - want[0]).abs() <= bound[0]).all()), b
