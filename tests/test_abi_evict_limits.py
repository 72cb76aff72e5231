"""Rows of a cache that mq_kv_evict counts in 32 bits: caches of almost 2^31 are refused, before any CUDA call. (Loops over
rows step by up to some thousand past the last.)"""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _call(L, cap, dst_cap, in_place=False):
    def kv(rows, base):
        return mq.CKV(base, base + (1 << 45), 0, 8, 0, 0, 1, rows, 1, 8)
    src = kv(cap, 1 << 46)
    dst = src if in_place else kv(dst_cap, 1 << 44)
    return L.mq_kv_evict(ctypes.byref(src), 16, 1 << 40, 4, 1, ctypes.byref(dst), 16, None, 1 << 41, None)


@pytest.mark.parametrize("cap,dst_cap,in_place", [(BIG, 10, False), (100, BIG, False), (BIG, BIG, True), (BIG - 5000, 10, False),
                                                  (100, BIG - 5000, False)])
def test_caches_of_almost_2_31_rows_are_refused(L, cap, dst_cap, in_place):
    assert _call(L, cap, dst_cap, in_place) == mq.MQ_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
def test_large_caches_are_taken(L):
    assert _call(L, 1 << 30, 1 << 30) == mq.MQ_ERR_ARCH and _call(L, (1 << 31) - (1 << 16), 10) == mq.MQ_ERR_ARCH
