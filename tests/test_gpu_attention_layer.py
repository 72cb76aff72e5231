"""The attention half of a layer from hidden state to hidden state (examples/attention_layer.py) against a
plain 64-bit form that starts from the products' own f32 outputs: prompt, decode steps past several
evictions, in lock step."""
import importlib.util
import os

import pytest
import torch

from quant_int8_quantized_gb300 import mq, synth
from tests import _attn_ref as R
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer_runs_and_stays_within_its_caches(example):
    layer = example.AttentionLayer(hidden=512, Hq=8, Hkv=2, D=64, batch=3, prefix_cap=80, cap=24, keep=10, recent=3, seed=3)
    y = layer.prompt(synth.normal((70, 512), 1, "p", device="cuda"))
    assert y.shape == (70, 512) and bool(y.isfinite().all())
    for t in range(60):
        y = layer.step(synth.normal((3, 512), 2, f"s{t}", device="cuda"))
        assert bool(y.isfinite().all())
        assert layer.length.tolist() == [layer.filled] * 3 and layer.filled <= 24
    assert layer.position.tolist() == [130] * 3
    assert mq.mq_device_status() == mq.MQ_OK


def test_each_call_of_a_step_against_64_bits(example, monkeypatch):
    """Every attention and eviction of 40 steps, checked from the arguments that the layer passes: the keys kept
    are those of the summed weights, and the outputs those of the keys kept."""
    layer = example.AttentionLayer(hidden=512, Hq=4, Hkv=2, D=64, batch=2, prefix_cap=40, cap=16, keep=8, recent=2, seed=5)
    layer.prompt(synth.normal((33, 512), 1, "p2", device="cuda"))
    attn, evict = mq.mq_attn_prefix, mq.mq_kv_evict
    seen = {"attn": 0, "evict": 0}

    def checked_attn(q, prefix, own, n, out, score=None, score_out=None, **kw):
        before = score.clone()
        attn(q, prefix, own, n, out, score=score, score_out=score_out, **kw)
        (o, _, s), (bo, _, bs) = R.attention(q, prefix.k[0], prefix.v[0], own.k, own.v, n.tolist(), 64 ** -0.5,
                                             torch.float32, before)
        assert bool(((out.double() - o).abs() <= bo).all())
        for b, m in enumerate(n.tolist()):
            assert bool(((score_out[b, :, :m].double() - s[b, :, :m]).abs() <= bs[b, :, :m]).all())
        seen["attn"] += 1

    def checked_evict(src, n, score, keep, recent, dst, n_out, score_out, index):
        want = [[R.evict(score[b, h].tolist(), int(n[b]), keep, recent) for h in range(2)] for b in range(2)]
        k = src.k.clone()
        evict(src, n, score, keep, recent, dst, n_out, score_out, index)
        for b in range(2):
            for h in range(2):
                assert index[b, h, :keep].tolist() == want[b][h]
                assert torch.equal(dst.k[b, :keep, h], k[b, want[b][h], h])
        seen["evict"] += 1

    monkeypatch.setattr(example.mq, "mq_attn_prefix", checked_attn)
    monkeypatch.setattr(example.mq, "mq_kv_evict", checked_evict)
    for t in range(40):
        layer.step(synth.normal((2, 512), 7, f"t{t}", device="cuda"))
    assert seen == {"attn": 40, "evict": 3}
