"""mq_qk_norm_rope refuses an output over its inputs, before any CUDA call (the output's rows are half as wide: a block would
write over another token's heads)."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

BASE = 1 << 30


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _call(L, M, q, k, v, stride, out, cache=1 << 33):
    x = mq.CQKV(q, k, v, stride, stride, stride, None, None, None, None, None, M, 4, 0, 0, 0, 1e-6)
    kv = mq.CKV(cache, cache + (1 << 32), 64 * 128, 128, 64, 0, 1, 64, 2, 64)
    return L.mq_qk_norm_rope(ctypes.byref(x), out, ctypes.byref(kv), None, None)


@pytest.mark.parametrize("M", [1, 2, 50])
@pytest.mark.parametrize("out", [0, 16, 1008, -496, 1536])
def test_queries_over_inputs_are_refused(L, M, out):
    """q, k and v side by side in rows of 512 floats (4 + 2 + 2 heads of 64)."""
    rc = _call(L, M, BASE, BASE + 1024, BASE + 1536, 512, BASE + out)
    assert rc == mq.MQ_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
@pytest.mark.parametrize("M,out", [(1, 2048), (1, -512), (50, 50 * 2048), (50, -50 * 512), (1, None)])
def test_queries_beside_inputs_are_taken(L, M, out):
    rc = _call(L, M, BASE if out is not None else None, BASE + 1024, BASE + 1536, 512, BASE + out if out is not None else None)
    assert rc == mq.MQ_ERR_ARCH
