"""Host-side checks of the calls on 4-bit caches and pages that need no GPU: what they refuse before any CUDA call,
no-ops, sizes."""
import ctypes

import pytest

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

FAR = 1 << 40


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _kv4(**kw):
    a = dict(pages=FAR, page_stride=64 // 16 * 2 * 17 * 128, table=16, table_stride=4, n=2, width=4, n_pages=10, page_rows=64, heads=2,
             dim=128) | kw
    return mq.CKV4(*a.values())


def _qkv(**kw):
    a = dict(q=16, k=16, v=16, q_stride=512, k_stride=256, v_stride=256, wq=None, wk=None, inv_freq=16, axis=None, pos=16,
             M=3, Hq=4, n_pairs=32, n_axes=1, interleaved=0, eps=1e-6) | kw
    return mq.CQKV(*a.values())


BAD = [(dict(n=-1), mq.MQ_ERR_SHAPE), (dict(width=-1), mq.MQ_ERR_SHAPE), (dict(n_pages=-1), mq.MQ_ERR_SHAPE),
       (dict(page_rows=8), mq.MQ_ERR_SHAPE), (dict(page_rows=48), mq.MQ_ERR_SHAPE), (dict(page_rows=2048), mq.MQ_ERR_SHAPE),
       (dict(heads=0), mq.MQ_ERR_SHAPE), (dict(dim=80), mq.MQ_ERR_SHAPE), (dict(dim=32), mq.MQ_ERR_SHAPE),
       (dict(page_stride=64 // 16 * 2 * 17 * 128 - 16), mq.MQ_ERR_SHAPE), (dict(page_stride=64 // 16 * 2 * 17 * 128 + 8), mq.MQ_ERR_SHAPE),
       (dict(table_stride=3), mq.MQ_ERR_SHAPE), (dict(width=1 << 26, table_stride=1 << 26), mq.MQ_ERR_SHAPE)]
BAD_POINTERS = [(dict(pages=None), mq.MQ_ERR_NULL), (dict(table=None), mq.MQ_ERR_NULL), (dict(pages=FAR + 8), mq.MQ_ERR_ALIGN),
                (dict(table=20), mq.MQ_ERR_ALIGN)]


def test_page_bytes(L):
    assert mq.mq_kv4_page_bytes(64, 8, 128) == 64 * 8 * 136
    assert mq.mq_kv4_page_bytes(16, 1, 96) == 16 * 102
    for bad in ((8, 1, 128), (24, 1, 128), (2048, 1, 128), (64, 0, 128), (64, 1, 120), (0, 1, 64)):
        assert mq.mq_kv4_page_bytes(*bad) == 0


def test_fill_refuses(L):
    def call(x=None, type=0, turn=1.0, out=1 << 30, cache=None, seq=None, row=16):
        return L.mq_qk_norm_rope_kv4(ctypes.byref(x or _qkv()), type, turn, out, ctypes.byref(cache or _kv4()), seq, row, None)

    assert L.mq_qk_norm_rope_kv4(None, 0, 1.0, 16, ctypes.byref(_kv4()), None, 16, None) == mq.MQ_ERR_NULL
    assert L.mq_qk_norm_rope_kv4(ctypes.byref(_qkv()), 0, 1.0, 16, None, None, 16, None) == mq.MQ_ERR_NULL
    for bad, status in BAD + BAD_POINTERS:
        assert call(cache=_kv4(**bad)) == status, bad
    for bad, status in ((dict(M=-1), mq.MQ_ERR_SHAPE), (dict(n_pairs=65), mq.MQ_ERR_SHAPE), (dict(n_pairs=-1), mq.MQ_ERR_SHAPE),
                        (dict(n_axes=0), mq.MQ_ERR_SHAPE), (dict(n_axes=9), mq.MQ_ERR_SHAPE), (dict(Hq=-1), mq.MQ_ERR_SHAPE),
                        (dict(q_stride=508), mq.MQ_ERR_SHAPE), (dict(k_stride=258), mq.MQ_ERR_SHAPE), (dict(q=20), mq.MQ_ERR_ALIGN),
                        (dict(v=24), mq.MQ_ERR_ALIGN), (dict(inv_freq=None), mq.MQ_ERR_NULL), (dict(pos=None), mq.MQ_ERR_NULL),
                        (dict(wq=17), mq.MQ_ERR_ALIGN), (dict(axis=1), mq.MQ_ERR_ALIGN)):
        assert call(_qkv(**bad)) == status, bad
    for bad, status in ((dict(type=2), mq.MQ_ERR_TYPE), (dict(turn=float("nan")), mq.MQ_ERR_SHAPE),
                        (dict(turn=float("inf")), mq.MQ_ERR_SHAPE), (dict(out=None), mq.MQ_ERR_NULL), (dict(row=None), mq.MQ_ERR_NULL),
                        (dict(out=8), mq.MQ_ERR_ALIGN), (dict(seq=4), mq.MQ_ERR_ALIGN), (dict(row=4), mq.MQ_ERR_ALIGN)):
        assert call(**bad) == status, bad
    # outputs over inputs or over one another
    assert call(out=16) == mq.MQ_ERR_SHAPE
    assert call(_qkv(k=FAR + 160)) == mq.MQ_ERR_SHAPE
    assert call(out=FAR + 10 * 64 // 16 * 2 * 17 * 128 - 16) == mq.MQ_ERR_SHAPE
    assert call(_qkv(M=0)) == mq.MQ_OK


def test_read_refuses(L):
    def kv(**kw):
        a = dict(k=16, v=1 << 30, seq=70 * 256, row=256, head=128, type=0, n=2, cap=70, heads=2, dim=128) | kw
        return mq.CKV(*a.values())

    def call(src=None, n=16, dst=None):
        return L.mq_kv4_read(ctypes.byref(src or _kv4()), n, ctypes.byref(dst or kv()), None)

    for bad, status in BAD + BAD_POINTERS:
        assert call(src=_kv4(**bad)) == status, bad
    for bad, status in ((dict(type=2), mq.MQ_ERR_TYPE), (dict(n=3), mq.MQ_ERR_SHAPE), (dict(heads=1), mq.MQ_ERR_SHAPE),
                        (dict(dim=64), mq.MQ_ERR_SHAPE), (dict(row=200), mq.MQ_ERR_SHAPE), (dict(k=None), mq.MQ_ERR_NULL),
                        (dict(v=20), mq.MQ_ERR_ALIGN), (dict(v=FAR), mq.MQ_ERR_SHAPE), (dict(k=FAR - 256), mq.MQ_ERR_SHAPE)):
        assert call(dst=kv(**bad)) == status, bad
    assert call(n=None) == mq.MQ_ERR_NULL and call(n=4) == mq.MQ_ERR_ALIGN
    assert call(src=_kv4(n=0), dst=kv(n=0)) == mq.MQ_OK and call(dst=kv(cap=0)) == mq.MQ_OK
    assert call(src=_kv4(width=0)) == mq.MQ_OK


def test_attention_refuses(L):
    need = mq.mq_attn_kv4_ws_bytes(2, 1, 4, 2, 128, 256)
    assert need > 0 and need % 16 == 0

    def call(q=16, type=0, stride=512, B=2, T=1, Hq=4, cache=None, n=16, scale=0.125, out=1 << 30, out_type=0, lse=None, ws=16, size=None):
        return L.mq_attn_kv4(q, type, stride, B, T, Hq, ctypes.byref(cache or _kv4()), n, scale, out, out_type, lse, ws,
                             need if size is None else size, None)

    assert L.mq_attn_kv4(16, 0, 512, 2, 1, 4, None, 16, 0.1, 16, 0, None, 16, need, None) == mq.MQ_ERR_NULL
    for bad, status in BAD + BAD_POINTERS:
        assert call(cache=_kv4(**bad)) == status, bad
    for bad, status in ((dict(B=-1), mq.MQ_ERR_SHAPE), (dict(T=-1), mq.MQ_ERR_SHAPE), (dict(B=3), mq.MQ_ERR_SHAPE),
                        (dict(Hq=3), mq.MQ_ERR_SHAPE), (dict(Hq=0), mq.MQ_ERR_SHAPE), (dict(type=2), mq.MQ_ERR_TYPE),
                        (dict(out_type=1), mq.MQ_ERR_TYPE), (dict(out_type=3), mq.MQ_ERR_TYPE), (dict(stride=504), mq.MQ_ERR_SHAPE),
                        (dict(stride=516), mq.MQ_ERR_SHAPE), (dict(stride=1 << 40), mq.MQ_ERR_SHAPE), (dict(scale=float("inf")), mq.MQ_ERR_SHAPE),
                        (dict(scale=float("nan")), mq.MQ_ERR_SHAPE), (dict(q=None), mq.MQ_ERR_NULL), (dict(out=None), mq.MQ_ERR_NULL),
                        (dict(ws=None), mq.MQ_ERR_NULL), (dict(n=None), mq.MQ_ERR_NULL), (dict(q=18), mq.MQ_ERR_ALIGN),
                        (dict(out=24), mq.MQ_ERR_ALIGN), (dict(lse=4), mq.MQ_ERR_ALIGN), (dict(n=4), mq.MQ_ERR_ALIGN),
                        (dict(ws=8), mq.MQ_ERR_ALIGN), (dict(size=need - 1), mq.MQ_ERR_SCRATCH), (dict(out=32), mq.MQ_ERR_SHAPE),
                        (dict(out=FAR), mq.MQ_ERR_SHAPE)):
        assert call(**bad) == status, bad
    assert call(B=0, cache=_kv4(n=0)) == mq.MQ_OK and call(T=0) == mq.MQ_OK


def test_attention_workspace(L):
    ws = mq.mq_attn_kv4_ws_bytes
    assert ws(0, 1, 4, 2, 128, 10) == 0 and ws(2, 0, 4, 2, 128, 10) == 0 and ws(2, 1, 4, 3, 128, 10) == 0
    assert ws(2, 1, 4, 2, 80, 10) == 0 and ws(1 << 20, 1 << 10, 64, 8, 128, 16) == 0
    assert ws(1, 3314, 28, 4, 128, 4352) < 256 << 20
    assert ws(64, 512, 40, 8, 128, 32768) < 3 << 30          # in parts
    sizes = [ws(b, 1, 40, 8, 128, 4096) for b in (1, 2, 8, 64)]
    assert sizes == sorted(sizes)


def _pool(**kw):
    a = dict(data=FAR, page_bytes=160, page_stride=160, layer_stride=1600, layers=2, n_pages=10, page_rows=16) | kw
    return mq.CPool(*a.values())


BAD_POOL = [(dict(page_bytes=0), mq.MQ_ERR_SHAPE), (dict(page_bytes=168), mq.MQ_ERR_SHAPE), (dict(page_stride=144), mq.MQ_ERR_SHAPE),
            (dict(page_stride=168), mq.MQ_ERR_SHAPE), (dict(layer_stride=1584), mq.MQ_ERR_SHAPE), (dict(layer_stride=8), mq.MQ_ERR_SHAPE),
            (dict(layers=0), mq.MQ_ERR_SHAPE), (dict(n_pages=-1), mq.MQ_ERR_SHAPE), (dict(n_pages=(1 << 28) + 1), mq.MQ_ERR_SHAPE),
            (dict(page_rows=0), mq.MQ_ERR_SHAPE), (dict(data=None), mq.MQ_ERR_NULL), (dict(data=FAR + 8), mq.MQ_ERR_ALIGN)]


def test_pages_refuse(L):
    need = L.mq_pages_ws_bytes(ctypes.byref(_pool()), 3, 4)
    assert need > 0 and need % 16 == 0 and L.mq_pages_ws_bytes(ctypes.byref(_pool()), -1, 4) == 0
    assert L.mq_pages_ws_bytes(None, 1, 1) == 0 and L.mq_pages_ws_bytes(ctypes.byref(_pool(page_rows=0)), 1, 1) == 0

    def step(pool=None, table=1024, ln=16, n=2, width=4, frm=16, keep=None, add=16, table_out=4096, ln_out=64, m=3, status=16, ws=16,
             size=None):
        return L.mq_pages_next(ctypes.byref(pool or _pool()), table, ln, n, width, frm, keep, add, table_out, ln_out, m, status, ws,
                               need if size is None else size, None)

    def close(pool=None, table=1024, ln=16, n=2, width=4, table_out=4096, where=16, live=16, ws=16, size=None):
        return L.mq_pages_compact(ctypes.byref(pool or _pool()), table, ln, n, width, table_out, where, live, ws,
                                  need if size is None else size, None)

    for bad, status in BAD_POOL:
        assert step(pool=_pool(**bad)) == status and close(pool=_pool(**bad)) == status, bad
    for bad, status in ((dict(n=-1), mq.MQ_ERR_SHAPE), (dict(width=-1), mq.MQ_ERR_SHAPE), (dict(width=1 << 30), mq.MQ_ERR_SHAPE),
                        (dict(table=None), mq.MQ_ERR_NULL), (dict(ln=None), mq.MQ_ERR_NULL), (dict(ws=None), mq.MQ_ERR_NULL),
                        (dict(table_out=None), mq.MQ_ERR_NULL), (dict(table=4), mq.MQ_ERR_ALIGN), (dict(ws=8), mq.MQ_ERR_ALIGN),
                        (dict(table_out=1024 + 16), mq.MQ_ERR_SHAPE)):
        assert step(**bad) == status and close(**bad) == status, bad
    for bad, status in ((dict(m=-1), mq.MQ_ERR_SHAPE), (dict(frm=None), mq.MQ_ERR_SHAPE), (dict(status=None), mq.MQ_ERR_NULL),
                        (dict(ln_out=None), mq.MQ_ERR_NULL), (dict(add=4), mq.MQ_ERR_ALIGN), (dict(keep=4), mq.MQ_ERR_ALIGN),
                        (dict(size=need - 1), mq.MQ_ERR_SCRATCH), (dict(n=6, ln=64, ln_out=80), mq.MQ_ERR_SHAPE)):
        assert step(**bad) == status, bad
    for bad, status in ((dict(where=None), mq.MQ_ERR_NULL), (dict(live=None), mq.MQ_ERR_NULL), (dict(where=4), mq.MQ_ERR_ALIGN),
                        (dict(size=0), mq.MQ_ERR_SCRATCH)):
        assert close(**bad) == status, bad


def test_pool_layouts(L):
    """Layers of pages and pages of layers are fine; pages of one layer among another's are not."""
    def ws(**kw):
        return L.mq_pages_ws_bytes(ctypes.byref(_pool(**kw)), 1, 1)

    assert ws() > 0 and ws(layers=1, layer_stride=-1) > 0 and ws(n_pages=1, page_stride=0, layer_stride=160) > 0
    assert ws(page_stride=320, layer_stride=160) > 0 and ws(page_stride=320, layer_stride=176) == 0


def test_binding_wants_its_types(L):
    import torch
    t = torch.zeros((4, 100), dtype=torch.uint8)
    with pytest.raises(ValueError):
        mq.KV4(t, t.int(), 16, 1, 64)
    with pytest.raises(TypeError):
        mq.KV4([1], t, 16, 1, 64)
    with pytest.raises(ValueError):
        mq.Pool(t, 16)
    with pytest.raises(TypeError):
        mq.Pool(None, 16)
    with pytest.raises(TypeError):
        mq.mq_kv4_read(t, t, t)
    with pytest.raises(TypeError):
        mq.mq_attn_kv4(t, t, t, t)
    with pytest.raises(TypeError):
        mq.mq_pages_next(t, t, t, t, t, t)


def test_scaled_frequencies():
    import math

    import torch
    n, factor, trained = 64, 4.0, 4096
    freq, turn = mq.rope_freq_scaled(n, 10000.0, factor, trained, device="cpu")
    plain = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    turns = trained * plain / (2 * math.pi)
    assert abs(turn - (1 + 0.1 * math.log(4))) < 1e-12
    for i in range(n):
        r = float(freq[i].double() / plain[i])
        want = 1.0 if turns[i] >= 32 else 0.25 if turns[i] <= 1 else 0.25 + 0.75 * (float(turns[i]) - 1) / 31
        assert abs(r - want) <= 2.0 ** -24 * 1.01
    same, one = mq.rope_freq_scaled(n, 10000.0, device="cpu")
    assert one == 1.0 and torch.equal(same, mq.rope_freq(n, device="cpu"))


def test_other_devices_are_refused(monkeypatch):
    """The calls run on the current device: tensors that say they are on another are not handed on."""
    import types

    import torch

    def on(i):
        return types.SimpleNamespace(device=torch.device("cuda", i), get_device=lambda: i)

    monkeypatch.setattr(mq, "_device", lambda: 1)
    mq._here("call", on(1), None, on(1))
    with pytest.raises(ValueError, match="current device"):
        mq._here("call", on(1), on(0))
