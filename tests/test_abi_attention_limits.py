"""Limits of mq_attn_prefix, without a GPU: calls that a limit does not concern are taken (they end at a workspace of
no bytes, before any CUDA call), those past one are refused."""
import ctypes

import pytest
import torch

from quant_int8_quantized_gb300 import build as B
from quant_int8_quantized_gb300 import mq


@pytest.fixture(scope="module")
def L():
    B.build()
    return mq.lib()


def _kv(n, cap, heads=2, dim=64, k=16, v=16, seq=None, row=None):
    row = heads * dim if row is None else row
    return mq.CKV(k, v, max(cap, 1) * row if seq is None else seq, row, dim, 0, n, cap, heads, dim)


def _call(L, B, T, Hq, prefix=None, own=None, q=1 << 20, stride=None, out=1 << 30, out_type=0, score=None, score_out=None, size=0):
    D = (own or prefix).dim
    return L.mq_attn_prefix(q, Hq * D if stride is None else stride, B, T, Hq, ctypes.byref(prefix) if prefix else None,
                            ctypes.byref(own) if own else None, 16 if own else None, 0.125, out, out_type, None, score,
                            score_out, 16, size, None)


@pytest.mark.parametrize("B,Hkv,T", [(8192, 8, 1), (70000, 1, 1), (8192, 9, 5)])
def test_sequences_times_heads_are_limited_with_weights_only(L, B, Hkv, T):
    own = _kv(B, 100, Hkv)
    assert _call(L, B, T, 2 * Hkv, own=own) == mq.MQ_ERR_SCRATCH
    assert _call(L, B, T, 2 * Hkv, own=own, prefix=_kv(1, 50, Hkv)) == mq.MQ_ERR_SCRATCH
    assert _call(L, B, T, 2 * Hkv, own=own, score=16, score_out=16) == mq.MQ_ERR_SHAPE


BIG = (1 << 31) - 1


@pytest.mark.parametrize("B,T,Hq,prefix_cap", [(BIG, BIG, 4, 5), (BIG, 1 << 30, 2, 5), (1 << 16, 1 << 16, 1 << 16, 5), (1 << 30, 1, 2, 5),
                                               (1, 1, 2, BIG), (1, 64, 8, BIG - 100)])
def test_counts_past_32_bits_are_refused(L, B, T, Hq, prefix_cap):
    assert _call(L, B, T, Hq, prefix=_kv(1, prefix_cap, 2 if Hq % 2 == 0 else 1)) == mq.MQ_ERR_SHAPE


def test_a_cache_of_more_rows_than_can_be_counted_is_refused(L):
    assert _call(L, 1, 1, 2, own=_kv(1, BIG, 1)) == mq.MQ_ERR_SHAPE
    assert _call(L, 1, 64, 8, own=_kv(1, BIG - 100, 1)) == mq.MQ_ERR_SHAPE


@pytest.mark.parametrize("B,T,Hq,Hkv,P,cap,scores", [(8192, 1, 64, 8, 0, 1 << 22, False), (64, 1 << 14, 40, 8, 0, 1 << 24, True),
                                                     (1, 1 << 20, 64, 8, 1 << 24, 0, False), (8192, 1, 16, 8, 0, 100, True),
                                                     (70000, 1, 2, 1, 30, 0, True), (70000, 1, 2, 1, 30, 5, True)])
def test_sizes_that_a_call_refuses_have_no_workspace(L, B, T, Hq, Hkv, P, cap, scores):
    """With weights, a cache of no rows has none to add up: such a call is taken."""
    own, prefix = _kv(B, cap, Hkv, 64), _kv(1, P, Hkv, 64) if P else None
    rc = _call(L, B, T, Hq, prefix=prefix, own=own, score=16 if scores else None, score_out=16 if scores else None)
    assert rc == (mq.MQ_ERR_SCRATCH if cap == 0 and scores else mq.MQ_ERR_SHAPE)
    assert (mq.mq_attn_ws_bytes(B, T, Hq, Hkv, 64, P, cap, scores) > 0) == (rc == mq.MQ_ERR_SCRATCH)


@pytest.mark.parametrize("what", ["own sequences", "own rows", "prefix rows", "queries"])
def test_strides_past_what_a_copy_can_step_are_refused(L, what):
    """2^40 bytes and more between rows that both exist: no tensor map holds that."""
    own, prefix, stride = _kv(2, 10), _kv(1, 10), None
    if what == "own sequences":
        own = _kv(2, 10, seq=1 << 39)
    elif what == "own rows":
        own = _kv(2, 10, row=1 << 39, seq=128)
    elif what == "prefix rows":
        prefix = _kv(1, 10, row=1 << 39, seq=0)
    else:
        stride = 1 << 39
    assert _call(L, 2, 1, 4, prefix=prefix, own=own, stride=stride) == mq.MQ_ERR_SHAPE


def test_a_stride_that_nothing_steps_along_does_not_matter(L):
    own = _kv(1, 10, seq=1 << 40)
    assert _call(L, 1, 1, 4, own=own, stride=1 << 40) == mq.MQ_ERR_SCRATCH


ENOUGH = 1 << 40      # bytes of workspace: what follows is looked at last, before the device


@pytest.mark.parametrize("T,Hq,stride,out,out_type", [
    (1, 4, 256, 0, 0), (600, 28, 28 * 64, 0, 0), (600, 28, 28 * 64, 0, 2), (600, 4, 1024, 512, 0),      # over q, over its gaps and rows
    (600, 28, 28 * 64, 600 * 28 * 128 - 16, 0), (600, 28, 28 * 64, -(600 * 28 * 128) + 16, 0),          # over its end, over its start
    (1, 4, 256, -1008, 2), (2, 4, 1 << 20, (1 << 21) - 16, 0)])
def test_outputs_over_queries_are_refused(L, T, Hq, stride, out, out_type):
    """Blocks that are done write rows of out while others still read q."""
    q = 1 << 30
    rc = _call(L, 1, T, Hq, own=_kv(1, 700, 2 if Hq == 4 else 4), q=q, stride=stride, out=q + out, out_type=out_type, size=ENOUGH)
    assert rc == mq.MQ_ERR_SHAPE


@pytest.mark.parametrize("at", [16, 16 * 70, -16])
def test_weights_over_others_are_refused(L, at):
    score = 1 << 29
    rc = _call(L, 2, 1, 4, own=_kv(2, 100), q=1 << 20, out=1 << 30, score=score, score_out=score + at, size=ENOUGH)
    assert rc == mq.MQ_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: these calls get as far as the device")
@pytest.mark.parametrize("T,stride,out", [(1, 256, 512), (1, 256, -512), (2, 1 << 20, 512), (2, 1 << 20, (1 << 21) - 1024), (2, 256, 1024)])
def test_outputs_beside_queries_and_weights_in_place_are_taken(L, T, stride, out):
    """Also between two rows of q that lie far apart."""
    q, score = 1 << 30, 1 << 29
    for at in (0, 2 * 2 * 100 * 4, -2 * 2 * 100 * 4):
        rc = _call(L, 1, T, 4, own=_kv(1, 200), q=q, stride=stride, out=q + out, score=score, score_out=score + at, size=ENOUGH)
        assert rc == mq.MQ_ERR_ARCH
