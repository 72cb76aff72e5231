"""mq_pages_next and mq_pages_compact refuse outputs and workspaces over one another, over what is read, and over the pool, before any
CUDA call."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

POOL = 1 << 40
N, M, WIDTH, PAGES, SIZE, LAYERS = 6, 9, 40, 50, 160, 3


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _pool(**kw):
    a = dict(data=POOL, page_bytes=SIZE, page_stride=SIZE, layer_stride=PAGES * SIZE, layers=LAYERS, n_pages=PAGES, page_rows=16) | kw
    return mq.CPool(*a.values())


def _next(L, pool=None, **kw):
    """The arrays a MB apart, but for those that kw places."""
    pool = pool or _pool()
    need = L.mq_pages_ws_bytes(ctypes.byref(pool), M, WIDTH)
    a = {n: (i + 1) << 20 for i, n in enumerate(("table", "len", "frm", "keep", "add", "table_out", "len_out", "status", "ws"))} | kw
    return L.mq_pages_next(ctypes.byref(pool), a["table"], a["len"], N, WIDTH, a["frm"], a["keep"], a["add"], a["table_out"], a["len_out"],
                           M, a["status"], a["ws"], need, None)


def _compact(L, pool=None, **kw):
    pool = pool or _pool()
    need = L.mq_pages_ws_bytes(ctypes.byref(pool), N, WIDTH)
    a = {n: (i + 1) << 20 for i, n in enumerate(("table", "len", "table_out", "where", "live", "ws"))} | kw
    return L.mq_pages_compact(ctypes.byref(pool), a["table"], a["len"], N, WIDTH, a["table_out"], a["where"], a["live"], a["ws"], need, None)


TABLE, LEN, FRM, KEEP, ADD, OUT, LEN_OUT, STATUS, WS = ((i + 1) << 20 for i in range(9))
LAST = POOL + LAYERS * PAGES * SIZE - 16


@pytest.mark.parametrize("kw", [
    dict(status=TABLE), dict(status=LEN + 16), dict(status=ADD), dict(status=OUT + 4 * M * WIDTH - 16), dict(status=LEN_OUT + 32), dict(status=WS + 64),
    dict(ws=TABLE), dict(ws=OUT), dict(ws=STATUS), dict(ws=FRM), dict(ws=LEN - 160), dict(len_out=KEEP), dict(len_out=FRM), dict(len_out=ADD),
    dict(len_out=TABLE), dict(len_out=LEN + 16), dict(len_out=OUT), dict(table_out=TABLE + 16), dict(table_out=TABLE - 16), dict(table_out=ADD),
    dict(table_out=LEN), dict(table_out=KEEP - 16),
    dict(status=POOL), dict(ws=POOL - 16), dict(table_out=LAST), dict(len_out=LAST), dict(table=POOL), dict(add=LAST), dict(len=POOL + 32)])
def test_next_refuses(L, kw):
    assert _next(L, **kw) == mq.MQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [
    dict(live=TABLE), dict(live=LEN), dict(live=OUT - (1 << 20) * 3 + 16), dict(where=TABLE - 16), dict(where=LEN), dict(ws=TABLE + 32), dict(ws=LEN),
    dict(table_out=TABLE + 16), dict(table_out=LEN), dict(where=POOL), dict(live=LAST), dict(ws=LAST), dict(table_out=POOL), dict(len=POOL), dict(table=LAST),
    dict(where=1 << 30, live=(1 << 30) + 16), dict(ws=1 << 30, live=(1 << 30) + 16), dict(ws=1 << 30, where=1 << 30)])
def test_compact_refuses(L, kw):
    assert _compact(L, **kw) == mq.MQ_ERR_SHAPE


NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")


@NO_DEVICE
def test_others_are_taken(L):
    """In place, side by side, one array for several inputs, between a pool's pages."""
    assert _next(L) == mq.MQ_ERR_ARCH and _compact(L) == mq.MQ_ERR_ARCH
    for kw in (dict(table_out=TABLE), dict(len_out=LEN), dict(table_out=TABLE, len_out=LEN), dict(frm=ADD, keep=ADD), dict(keep=None, add=None),
               dict(status=LEN + 32), dict(status=OUT + 4 * M * WIDTH), dict(ws=LAST + 16), dict(table_out=POOL - 4 * M * WIDTH), dict(len=TABLE)):
        assert _next(L, **kw) == mq.MQ_ERR_ARCH, kw
    for kw in (dict(table_out=TABLE), dict(live=LEN + 32), dict(where=LAST + 16), dict(len=TABLE)):
        assert _compact(L, **kw) == mq.MQ_ERR_ARCH, kw
    # a slice of wider pages, and pages of layers: what lies between them is not the pool's
    wide = _pool(page_stride=SIZE + 64, layer_stride=PAGES * (SIZE + 64))
    assert _next(L, wide, status=POOL + SIZE) == mq.MQ_ERR_ARCH and _next(L, wide, status=POOL + SIZE + 64) == mq.MQ_ERR_SHAPE
    inner = _pool(page_stride=LAYERS * SIZE + 32, layer_stride=SIZE)
    assert _compact(L, inner, live=POOL + LAYERS * SIZE) == mq.MQ_ERR_ARCH and _compact(L, inner, live=POOL + SIZE) == mq.MQ_ERR_SHAPE
    one = _pool(n_pages=1, page_stride=0, layer_stride=SIZE)
    assert _next(L, one, status=POOL + LAYERS * SIZE) == mq.MQ_ERR_ARCH and _next(L, one, status=POOL + 2 * SIZE) == mq.MQ_ERR_SHAPE
    assert _next(L, _pool(n_pages=0), status=POOL) == mq.MQ_ERR_ARCH
