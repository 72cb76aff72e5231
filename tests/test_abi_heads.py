"""Host-side checks of the calls between attn_q|k|v and attn_o that need no GPU: what they refuse before any
CUDA call, no-ops, sizes."""
import ctypes

import pytest

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq

V = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _kv(k=16, v=16, n=2, cap=10, heads=2, dim=64, seq=None, row=None, head=None, type=0):
    row = heads * dim if row is None else row
    return mq.CKV(k, v, cap * row if seq is None else seq, row, dim if head is None else head, type, n, cap, heads, dim)


def _qkv(**kw):
    a = dict(q=16, k=16, v=16, q_stride=256, k_stride=128, v_stride=128, wq=None, wk=None, inv_freq=16, axis=None, pos=16,
             M=3, Hq=4, n_pairs=32, n_axes=1, interleaved=0, eps=1e-6) | kw
    return mq.CQKV(*a.values())


BAD_KV = [(dict(type=2), mq.MQ_ERR_TYPE), (dict(type=-1), mq.MQ_ERR_TYPE), (dict(n=-1), mq.MQ_ERR_SHAPE),
          (dict(cap=-1), mq.MQ_ERR_SHAPE), (dict(heads=0), mq.MQ_ERR_SHAPE), (dict(dim=60), mq.MQ_ERR_SHAPE),
          (dict(dim=264), mq.MQ_ERR_SHAPE), (dict(row=127), mq.MQ_ERR_SHAPE), (dict(row=120), mq.MQ_ERR_SHAPE),
          (dict(head=0), mq.MQ_ERR_SHAPE), (dict(seq=1272), mq.MQ_ERR_SHAPE), (dict(seq=-8), mq.MQ_ERR_SHAPE),
          (dict(seq=1 << 41), mq.MQ_ERR_SHAPE)]


def test_rope_refuses(L):
    fn = L.mq_qk_norm_rope

    def call(x, kv=None, out=16, slot=None):
        kv = kv or _kv()
        return fn(ctypes.byref(x) if x else None, V(out), ctypes.byref(kv), V(slot) if slot else None, None)

    assert call(None) == mq.MQ_ERR_NULL
    for bad, status in BAD_KV:
        assert call(_qkv(), _kv(**bad)) == status, bad
    for bad, status in ((dict(M=-1), mq.MQ_ERR_SHAPE), (dict(n_pairs=33), mq.MQ_ERR_SHAPE), (dict(n_pairs=-1), mq.MQ_ERR_SHAPE),
                        (dict(n_axes=0), mq.MQ_ERR_SHAPE), (dict(n_axes=9), mq.MQ_ERR_SHAPE), (dict(Hq=-1), mq.MQ_ERR_SHAPE),
                        (dict(q_stride=252), mq.MQ_ERR_SHAPE), (dict(k_stride=130), mq.MQ_ERR_SHAPE),
                        (dict(M=21), mq.MQ_ERR_SHAPE), (dict(q=20), mq.MQ_ERR_ALIGN), (dict(v=24), mq.MQ_ERR_ALIGN),
                        (dict(inv_freq=None), mq.MQ_ERR_NULL), (dict(pos=None), mq.MQ_ERR_NULL),
                        (dict(wq=17), mq.MQ_ERR_ALIGN), (dict(axis=1), mq.MQ_ERR_ALIGN)):
        assert call(_qkv(**bad)) == status, bad
    assert call(_qkv(), out=0) == mq.MQ_ERR_NULL and call(_qkv(), out=8) == mq.MQ_ERR_ALIGN
    assert call(_qkv(), _kv(k=None)) == mq.MQ_ERR_NULL and call(_qkv(), _kv(v=40)) == mq.MQ_ERR_ALIGN
    assert call(_qkv(), slot=4) == mq.MQ_ERR_ALIGN
    assert call(_qkv(M=0)) == mq.MQ_OK


def test_attention_refuses(L):
    fn = L.mq_attn_prefix
    need = mq.mq_attn_ws_bytes(2, 1, 4, 2, 64, 5, 10)
    assert need > 0 and need % 16 == 0

    def call(q=16, stride=256, B=2, T=1, Hq=4, prefix="own", own="own", n=16, scale=0.125, out=16, out_type=0, lse=None,
             score=None, score_out=None, ws=16, size=None):
        prefix = _kv(n=1, cap=5) if prefix == "own" else prefix
        own = _kv() if own == "own" else own
        return fn(q, stride, B, T, Hq, ctypes.byref(prefix) if prefix else None, ctypes.byref(own) if own else None, n,
                  scale, out, out_type, lse, score, score_out, ws, need if size is None else size, None)

    for bad, status in BAD_KV:
        assert call(own=_kv(**bad)) == status, bad
        if "n" not in bad and "seq" not in bad:
            assert call(prefix=_kv(**(dict(n=1, cap=5) | bad))) == status, bad
    for bad, status in (
            (dict(prefix=None, own=None), mq.MQ_ERR_NULL), (dict(B=-1), mq.MQ_ERR_SHAPE), (dict(T=-1), mq.MQ_ERR_SHAPE),
            (dict(B=3), mq.MQ_ERR_SHAPE), (dict(Hq=3), mq.MQ_ERR_SHAPE), (dict(Hq=0), mq.MQ_ERR_SHAPE),
            (dict(prefix=_kv(n=2, cap=5)), mq.MQ_ERR_SHAPE), (dict(prefix=_kv(n=1, cap=5, heads=1)), mq.MQ_ERR_SHAPE),
            (dict(prefix=_kv(n=1, cap=5, dim=128)), mq.MQ_ERR_SHAPE), (dict(prefix=_kv(n=1, cap=5, type=1)), mq.MQ_ERR_TYPE),
            (dict(own=_kv(dim=80), prefix=None), mq.MQ_ERR_SHAPE), (dict(out_type=1), mq.MQ_ERR_TYPE),
            (dict(out_type=3), mq.MQ_ERR_TYPE), (dict(stride=255), mq.MQ_ERR_SHAPE), (dict(stride=252), mq.MQ_ERR_SHAPE),
            (dict(scale=float("inf")), mq.MQ_ERR_SHAPE), (dict(scale=float("nan")), mq.MQ_ERR_SHAPE),
            (dict(q=None), mq.MQ_ERR_NULL), (dict(out=None), mq.MQ_ERR_NULL), (dict(ws=None), mq.MQ_ERR_NULL),
            (dict(n=None), mq.MQ_ERR_NULL), (dict(score=16), mq.MQ_ERR_NULL), (dict(score_out=16), mq.MQ_ERR_NULL),
            (dict(q=18), mq.MQ_ERR_ALIGN), (dict(out=24), mq.MQ_ERR_ALIGN), (dict(lse=4), mq.MQ_ERR_ALIGN),
            (dict(n=4), mq.MQ_ERR_ALIGN), (dict(score=4, score_out=16), mq.MQ_ERR_ALIGN), (dict(size=need - 1), mq.MQ_ERR_SCRATCH),
            (dict(own=_kv(k=None)), mq.MQ_ERR_NULL), (dict(own=_kv(v=20)), mq.MQ_ERR_ALIGN)):
        assert call(**bad) == status, bad
    assert call(B=0, own=_kv(n=0)) == mq.MQ_OK and call(T=0) == mq.MQ_OK


def test_workspace_sizes(L):
    assert mq.mq_attn_ws_bytes(0, 1, 4, 2, 64, 5, 10) == 0 and mq.mq_attn_ws_bytes(2, 1, 4, 3, 64, 5, 10) == 0
    assert mq.mq_attn_ws_bytes(2, 1, 4, 2, 80, 5, 10) == 0
    plain, scored = (mq.mq_attn_ws_bytes(2, 1, 4, 2, 64, 5, 10, s) for s in (False, True))
    assert scored >= plain + 2 * 4 * 10 * 4
    sizes = [mq.mq_attn_ws_bytes(b, 1, 40, 8, 128, 4096, 1024) for b in (1, 2, 8, 64)]
    assert sizes == sorted(sizes)
    assert mq.mq_attn_ws_bytes(1, 3314, 28, 4, 128, 1000, 3314) < 256 << 20
    # counts that would not fit int32 have no size, and are refused
    assert mq.mq_attn_ws_bytes(1 << 20, 1 << 10, 64, 8, 128, 0, 10) == 0


def test_evict_refuses(L):
    fn = L.mq_kv_evict

    def call(src=None, n=16, score=16, keep=4, recent=1, dst=None, n_out=16, score_out=None, index=16):
        src, dst = src or _kv(), dst or _kv(k=1 << 20, v=1 << 21, cap=5)
        return fn(ctypes.byref(src), n, score, keep, recent, ctypes.byref(dst), n_out, score_out, index, None)

    for bad, status in BAD_KV:
        assert call(src=_kv(**bad)) == status and call(dst=_kv(**bad)) == status, bad
    far = dict(k=1 << 20, v=1 << 21)
    for bad, status in (
            (dict(dst=_kv(type=1, cap=5, **far)), mq.MQ_ERR_TYPE), (dict(dst=_kv(n=1, cap=5, **far)), mq.MQ_ERR_SHAPE),
            (dict(dst=_kv(heads=1, cap=5, **far)), mq.MQ_ERR_SHAPE), (dict(dst=_kv(dim=128, cap=5, **far)), mq.MQ_ERR_SHAPE),
            (dict(keep=6), mq.MQ_ERR_SHAPE), (dict(recent=5), mq.MQ_ERR_SHAPE), (dict(recent=-1), mq.MQ_ERR_SHAPE),
            (dict(keep=-1, recent=-1), mq.MQ_ERR_SHAPE), (dict(n=None), mq.MQ_ERR_NULL), (dict(n_out=None), mq.MQ_ERR_NULL),
            (dict(score=None), mq.MQ_ERR_NULL), (dict(index=None), mq.MQ_ERR_NULL), (dict(index=4), mq.MQ_ERR_ALIGN),
            (dict(score=8), mq.MQ_ERR_ALIGN), (dict(src=_kv(k=None)), mq.MQ_ERR_NULL),
            (dict(dst=_kv(cap=5)), mq.MQ_ERR_SHAPE), (dict(dst=_kv(k=1 << 20, v=16, cap=5)), mq.MQ_ERR_SHAPE),
            (dict(src=_kv(k=16, v=1 << 16), dst=_kv(k=16, v=1 << 20)), mq.MQ_ERR_SHAPE),
            (dict(score=16, score_out=32), mq.MQ_ERR_SHAPE)):
        assert call(**bad) == status, bad
    assert call(src=_kv(n=0), dst=_kv(n=0, cap=5, **far)) == mq.MQ_OK


def test_status_names(L):
    assert mq.status_str(mq.MQ_ERR_TYPE).startswith("MQ_ERR_TYPE")


def test_binding_wants_cuda_tensors(L):
    import torch
    t = torch.zeros((1, 4, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        mq.KV(t, t)
    with pytest.raises(TypeError):
        mq.KV([1], [2])
