"""The attention kernels' failure path, without a GPU fault: a test build (50 ms wait limit) whose first block
leaves out a copy, so that the bounded waits for it run out. The kernel must return, the status say so
once, and the next call, with the copy made, be right."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def inject():
    require_gpu()
    own = mq.lib()
    L = mq._load(B.build_variant("attn_inject", ["MQ_TEST_INJECT", "MQ_WAIT_LIMIT_NS=50000000ull", "MQ_FEW_BYTES=8000000"]))
    L.mq_test_inject_attn.restype, L.mq_test_inject_attn.argtypes = ctypes.c_int, [ctypes.c_int]
    mq._lib = L
    yield L.mq_test_inject_attn
    assert L.mq_test_inject_attn(0) == mq.MQ_OK
    mq._lib = own


@pytest.mark.parametrize("bit,T", [(1, 600), (2, 1), (2, 20)])
def test_wait_runs_out_is_reported_and_forgotten(inject, bit, T):
    Bt, Hq, Hkv, D, cap = 2, 8, 2, 128, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    q, k, v = (torch.randn(s, generator=g, device="cuda").half() for s in ((Bt, T, Hq, D), (Bt, cap, Hkv, D), (Bt, cap, Hkv, D)))
    n = torch.tensor([700, 650], dtype=torch.int32, device="cuda")
    out = torch.zeros((Bt, T, Hq, D), dtype=torch.float16, device="cuda")
    assert mq.mq_device_status() == mq.MQ_OK
    ws = mq.attn_workspace(Bt, T, Hq, Hkv, D, 0, cap)
    ws.fill_(0x7F)                                      # entries that are not written must not be followed
    assert inject(bit) == mq.MQ_OK
    mq.mq_attn_prefix(q, None, mq.KV(k, v), n, out, ws=ws)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_ERR_DEVICE
    assert mq.mq_device_status() == mq.MQ_OK
    assert inject(0) == mq.MQ_OK
    mq.mq_attn_prefix(q, None, mq.KV(k, v), n, out, ws=ws)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    only = [0, T // 2, T - 1]
    want, bound = R.attention(q, None, None, k, v, [700, 650], D ** -0.5, torch.float16, only=only)
    assert bool(((out[:, only].double() - want[0][:, only]).abs() <= bound[0][:, only]).all())
