"""mq_attn_prefix at the edges of what it takes. Every test runs on the library as it is and on a test build that sends
calls of any size to the tensor-core kernel."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


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


def test_strides_that_nothing_steps_along():
    """One sequence, one query: neither has a next one whose place could matter."""
    Hq, Hkv, D, P, cap = 4, 2, 64, 40, 90
    q, k, v = (_rand((1, n, h, D), F16, i) for i, (n, h) in enumerate(((1, Hq), (cap, Hkv), (cap, Hkv))))
    pk, pv = _rand((1, P, Hkv, D), F16, 3), _rand((1, P, Hkv, D), F16, 4)
    own, pre = mq.KV(k, v), mq.KV(pk, pv)
    own._c.seq_stride = pre._c.seq_stride = 1 << 40
    n, out = torch.tensor([77], dtype=torch.int32, device="cuda"), torch.empty((1, 1, Hq, D), device="cuda")
    ws = mq.attn_workspace(1, 1, Hq, Hkv, D, P, cap)
    rc = mq.lib().mq_attn_prefix(q.data_ptr(), 1 << 40, 1, 1, Hq, ctypes.byref(pre._c), ctypes.byref(own._c), n.data_ptr(), D ** -0.5,
                                 out.data_ptr(), 2, None, None, None, ws.data_ptr(), ws.numel(),
                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == mq.MQ_OK
    want, bound = R.attention(q, pk[0], pv[0], k, v, [77], D ** -0.5, F32)
    assert bool(((out.double() - want[0]).abs() <= bound[0]).all())


@pytest.mark.parametrize("T", [1, 40, 600])
def test_outputs_over_queries(T):
    """Over the queries: refused, whichever kernel would run. Beside them in one allocation: right."""
    Hq, Hkv, D, cap = 28, 4, 64, T + 100
    both = _rand((1, T, 2 * Hq, D), F16, 1)
    q, beside = both[:, :, :Hq].contiguous(), _rand((2, 1, T, Hq, D), F16, 1)
    k, v = _rand((1, cap, Hkv, D), F16, 2), _rand((1, cap, Hkv, D), F16, 3)
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    own = mq.KV(k, v)
    over = [(q, q)]
    if T > 1:                                          # rows of the other heads, between which the output has no place
        over.append((both[:, :, Hq:], both.view(-1)[:T * Hq * D]))
    for x, out in over:
        before = x.clone()
        with pytest.raises(mq.MQError) as e:
            mq.mq_attn_prefix(x, None, own, n, out)
        assert e.value.status == mq.MQ_ERR_SHAPE and torch.equal(x, before)
    beside[0] = q
    mq.mq_attn_prefix(beside[0], None, own, n, beside[1])
    only = [0, T // 2, T - 1]
    want, bound = R.attention(q, None, None, k, v, [cap], D ** -0.5, F16, only=only)
    assert bool(((beside[1][:, only].double() - want[0][:, only]).abs() <= bound[0][:, only]).all())
