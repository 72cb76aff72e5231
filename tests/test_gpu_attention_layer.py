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


def test_lock_step_with_64_bits(example, monkeypatch):
    """Prompt and 40 decode steps beside a layer of its own kind, which knows positions, rows, lengths, scores and
    evictions by itself and computes in 64 bits from the products' f32 outputs. What the layer rounds to 16 bits or sums
    up in f32 is checked and then taken over, so that both stay in step."""
    B, Hq, Hkv, D, cap, keep, recent, T = 2, 4, 2, 64, 16, 8, 2, 33
    layer = example.AttentionLayer(hidden=512, Hq=Hq, Hkv=Hkv, D=D, batch=B, prefix_cap=40, cap=cap, keep=keep, recent=recent, seed=11)
    saw, rope, quant = {}, mq.mq_qk_norm_rope, mq.mq_quantize_q8

    def watch_rope(q, k, v, q_out, *a, **kw):
        saw.update(q=q.clone(), k=k.clone(), v=v.clone())
        saw["q16"] = rope(q, k, v, q_out, *a, **kw)
        return saw["q16"]

    def watch_quant(x, plane):
        saw["o"] = x.clone()
        return quant(x, plane)

    monkeypatch.setattr(example.mq, "mq_qk_norm_rope", watch_rope)
    monkeypatch.setattr(example.mq, "mq_quantize_q8", watch_quant)

    def inside(got, want, bound):
        return bool(((got.double() - want).abs() <= bound).all())

    def turned(positions):
        pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
        return [R.rope(saw[x], w, 1e-6, pos, layer.freq, None, 1, False, layer.dtype) for x, w in (("q", layer.q_norm), ("k", layer.k_norm))]

    layer.prompt(synth.normal((T, 512), 1, "lock.p", device="cuda"))
    (wq, bq), (wk, bk) = turned(list(range(T)))
    pk, pv = layer.prefix.k[0, :T].clone(), layer.prefix.v[0, :T].clone()
    assert inside(saw["q16"], wq, bq) and inside(pk, wk, bk) and torch.equal(pv, saw["v"].to(layer.dtype))
    (o, _, _), (bo, _, _) = R.attention(saw["q16"][None], None, None, pk[None], pv[None], [T], D ** -0.5, torch.float32)
    assert inside(saw["o"].view(1, T, Hq, D), o, bo)

    # caches, one head at a time: rows kept [rows, D] and their scores
    ks = [[torch.empty((0, D), dtype=layer.dtype, device="cuda") for _ in range(Hkv)] for _ in range(B)]
    vs = [[x.clone() for x in row] for row in ks]
    sc = [[torch.empty((0,), device="cuda") for _ in range(Hkv)] for _ in range(B)]
    evictions = 0
    for t in range(40):
        if len(ks[0][0]) == cap:
            evictions += 1
            for b in range(B):
                for h in range(Hkv):
                    rows = R.evict(sc[b][h].tolist(), cap, keep, recent)
                    ks[b][h], vs[b][h], sc[b][h] = (x[b][h][rows] for x in (ks, vs, sc))
        layer.step(synth.normal((B, 512), 2, f"lock.{t}", device="cuda"))
        (wq, bq), (wk, bk) = turned([T + t] * B)
        n = len(ks[0][0]) + 1
        assert layer.length.tolist() == [n] * B and layer.position.tolist() == [T + t + 1] * B
        assert inside(saw["q16"], wq, bq)
        k, v = layer.own.k[:, :n].clone(), layer.own.v[:, :n].clone()
        score = torch.zeros((B, Hkv, n), device="cuda")
        for b in range(B):
            for h in range(Hkv):
                assert torch.equal(k[b, :n - 1, h], ks[b][h]) and torch.equal(v[b, :n - 1, h], vs[b][h]), (t, b, h)
                assert inside(k[b, n - 1, h], wk[b, h], bk[b, h]) and torch.equal(v[b, n - 1, h], saw["v"][b, h].to(layer.dtype))
                score[b, h, :n - 1] = sc[b][h]
        (o, _, s), (bo, _, bs) = R.attention(saw["q16"].view(B, 1, Hq, D), pk, pv, k, v, [n] * B, D ** -0.5, torch.float32, score)
        assert inside(saw["o"].view(B, 1, Hq, D), o, bo) and inside(layer.score[:, :, :n], s, bs)
        for b in range(B):
            for h in range(Hkv):
                ks[b][h], vs[b][h], sc[b][h] = k[b, :, h], v[b, :, h], layer.score[b, h, :n].clone()
    assert evictions == 3
