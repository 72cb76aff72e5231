"""Strides of a size that no memory has: refused where something steps along them, of no matter for one token; never a process that
ends (bytes from token to token that wrap to 0 were divided by)."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

HUGE = [(1 << 40) + 4, 1 << 59, 1 << 60, 1 << 61, 1 << 62, (1 << 63) - 4]


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _calls(L, M, which, stride):
    st = {n: stride if n == which else 512 for n in "qkv"}
    x = mq.CQKV(1 << 30, 1 << 31, 1 << 33, st["q"], st["k"], st["v"], None, None, None, None, None, M, 4, 0, 0, 0, 1e-6)
    kv4 = mq.CKV4(1 << 40, 8 * 17 * 128, 16, 4, 2, 4, 10, 64, 2, 128)
    kv = mq.CKV(1 << 34, 1 << 35, 64 * 256, 256, 128, 0, 1, 64, 2, 128)
    return (L.mq_qk_norm_rope_kv4(ctypes.byref(x), 0, 1.0, 1 << 32, ctypes.byref(kv4), None, 16, None),
            L.mq_qk_norm_rope(ctypes.byref(x), 1 << 32, ctypes.byref(kv), None, None))


@pytest.mark.parametrize("stride", HUGE)
@pytest.mark.parametrize("which", "qkv")
def test_several_tokens_are_refused(L, which, stride):
    assert _calls(L, 2, which, stride) == (mq.MQ_ERR_SHAPE, mq.MQ_ERR_SHAPE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
@pytest.mark.parametrize("stride", HUGE)
@pytest.mark.parametrize("which", "qkv")
def test_one_token_is_taken(L, which, stride):
    assert _calls(L, 1, which, stride) == (mq.MQ_ERR_ARCH, mq.MQ_ERR_ARCH)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
@pytest.mark.parametrize("stride", [1 << 60, 1 << 61, 1 << 62, (1 << 63) - 8])
def test_one_query_is_taken(L, stride):
    cache = mq.CKV4(1 << 40, 8 * 17 * 128, 16, 4, 1, 4, 10, 64, 2, 128)
    need = mq.mq_attn_kv4_ws_bytes(1, 1, 4, 2, 128, 256)
    assert L.mq_attn_kv4(1 << 30, 0, stride, 1, 1, 4, ctypes.byref(cache), 16, 0.1, 1 << 32, 0, None, 1 << 20, need, None) == mq.MQ_ERR_ARCH
