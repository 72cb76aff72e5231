"""Caches whose pages lie among other layers' pages: what begins behind the pool, or between a layer's pages, is not over them."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

POOL, LAYERS, PAGES, HEADS, D = 1 << 40, 28, 10, 2, 128
SIZE = 4 * HEADS * 17 * D                    # pages of 64 rows
END = POOL + PAGES * LAYERS * SIZE           # [page][layer][bytes]


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _cache(layer, data=POOL):
    return mq.CKV4(data + layer * SIZE, LAYERS * SIZE, 16, 4, 2, 4, PAGES, 64, HEADS, D)


def _fill(L, layer, q=1 << 30, k=1 << 31, out=1 << 32):
    x = mq.CQKV(q, k, k + 1024, 512, 512, 512, None, None, None, None, None, 3, 4, 0, 0, 0, 1e-6)
    return L.mq_qk_norm_rope_kv4(ctypes.byref(x), 0, 1.0, out, ctypes.byref(_cache(layer)), None, 16, None)


def _read(L, layer, k=1 << 32, v=1 << 33):
    dst = mq.CKV(k, v, 70 * 256, 256, 128, 0, 2, 70, HEADS, D)
    return L.mq_kv4_read(ctypes.byref(_cache(layer)), 16, ctypes.byref(dst), None)


def _attend(L, layer, out=1 << 32):
    need = mq.mq_attn_kv4_ws_bytes(2, 1, 4, HEADS, D, 256)
    return L.mq_attn_kv4(1 << 30, 0, 512, 2, 1, 4, ctypes.byref(_cache(layer)), 16, 0.1, out, 0, None, 1 << 20, need, None)


LAST = [(0, END - LAYERS * SIZE + SIZE - 16), (LAYERS - 1, END - 16), (3, POOL + 3 * SIZE), (5, POOL + 6 * SIZE - 16)]


@pytest.mark.parametrize("layer,at", LAST)
def test_over_a_page_is_refused(L, layer, at):
    for rc in (_fill(L, layer, out=at), _read(L, layer, k=at), _read(L, layer, v=at), _attend(L, layer, out=at), _fill(L, layer, q=at),
               _fill(L, layer, k=at)):
        assert rc == mq.MQ_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
@pytest.mark.parametrize("layer", [0, 5, LAYERS - 1])
def test_behind_the_pool_is_taken(L, layer):
    """A pool's layers side by side in each page: the last layer's pages end where the pool does."""
    for rc in (_fill(L, layer, out=END), _read(L, layer, k=END), _read(L, layer, v=END), _attend(L, layer, out=END), _fill(L, layer, q=END),
               _fill(L, layer, k=END)):
        assert rc == mq.MQ_ERR_ARCH
