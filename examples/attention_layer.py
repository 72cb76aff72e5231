"""The attention half of a decoder layer on quantized weights, from hidden state to hidden state:

    RMSNorm -> q8 plane -> attn_q|k|v products -> head norms, rotation, cache write
    -> attention over a shared prefix and each sequence's own cache -> q8 plane -> attn_o product

for prompts (GEMMs) and for decode steps of a batch (GEMVs), with caches of a fixed size: every decode step
adds up how much each key was attended to, and a cache that is full is cut to its most attended and its
latest rows.

    python examples/attention_layer.py        # a short run on synthetic weights
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quant_int8_quantized_gb300 import mq, synth  # noqa: E402


class AttentionLayer:
    """Weights of one layer (attn_q, attn_k, attn_o in q4_K, attn_v in q6_K) and the caches of `batch` sequences
    that share one prefix."""

    def __init__(self, hidden, Hq, Hkv, D, batch, prefix_cap, cap, keep, recent, seed=0, dtype=torch.float16,
                 rope_base=10000.0, device="cuda"):
        assert keep < cap and batch <= mq.MQ_GEMV_MAX_ROWS
        self.hidden, self.Hq, self.Hkv, self.D, self.batch = hidden, Hq, Hkv, D, batch
        self.cap, self.keep, self.recent, self.device, self.dtype = cap, keep, recent, device, dtype
        self.wq = synth.weights("q4k", Hq * D, hidden, seed, "layer.q", device)
        self.wk = synth.weights("q4k", Hkv * D, hidden, seed, "layer.k", device)
        wv = synth.weights("q6k", Hkv * D, hidden, seed, "layer.v", device)
        self.wv = mq.mq_prepack_q6k(wv, Hkv * D, hidden)
        self.wo = synth.weights("q4k", hidden, Hq * D, seed, "layer.o", device)
        self.norm = synth.normal((hidden,), seed, "layer.norm", 1.0, 0.1, device)
        self.q_norm = synth.normal((D,), seed, "layer.q_norm", 1.0, 0.1, device)
        self.k_norm = synth.normal((D,), seed, "layer.k_norm", 1.0, 0.1, device)
        self.freq = mq.rope_freq(D // 2, rope_base, device)
        # the prefix that all sequences share, and two sets of own caches: eviction moves rows from one to the other
        self.prefix = mq.KV.empty(1, prefix_cap, Hkv, D, dtype, device)
        self.prefix_len = 0
        self.own, self.spare = (mq.KV.empty(batch, cap, Hkv, D, dtype, device) for _ in range(2))
        self.score = torch.zeros((batch, Hkv, cap), device=device)
        self.spare_score = torch.zeros_like(self.score)
        self.index = torch.empty((batch, Hkv, cap), dtype=torch.int32, device=device)
        self.length = torch.zeros((batch,), dtype=torch.int32, device=device)
        self.position = torch.zeros((batch,), dtype=torch.int32, device=device)    # of the next token
        self.rows = torch.arange(batch, dtype=torch.int32, device=device) * cap
        self.filled = 0                                                           # rows of the fullest cache

    def _project(self, x, pos, cache, slot):
        """Queries [M, Hq, D] in 16 bits; keys and values of the M rows x go to the cache's rows `slot`."""
        M = x.shape[0]
        Nq, Nk = self.Hq * self.D, self.Hkv * self.D
        few = M <= mq.MQ_GEMV_MAX_ROWS
        plane = mq.Plane.empty(M, self.hidden, self.device, q8=few, op=not few)
        mq.mq_rms_quant(x, self.norm, 1e-6, plane)
        q, k, v = (torch.empty((M, n), device=self.device) for n in (Nq, Nk, Nk))
        if few:
            mq.mq_gemv_q4k(plane, self.wq, Nq, q)
            mq.mq_gemv_q4k(plane, self.wk, Nk, k)
            mq.mq_gemv_q6k_packed(plane, self.wv, Nk, v)
        else:
            mq.mq_gemm_q4k_pair(plane, self.wq, Nq, q, self.wk, Nk, k)
            mq.mq_gemm_q6k(plane, self.wv, Nk, v)
        out = torch.empty((M, self.Hq, self.D), dtype=self.dtype, device=self.device)
        heads = (lambda t, n: t.view(M, n, self.D))
        return mq.mq_qk_norm_rope(heads(q, self.Hq), heads(k, self.Hkv), heads(v, self.Hkv), out, cache, slot, pos,
                                  self.freq, wq=self.q_norm, wk=self.k_norm)

    def _output(self, o):
        """attn_o of the heads' outputs (f32 [M, Hq, D])."""
        M, K = o.shape[0], self.Hq * self.D
        few = M <= mq.MQ_GEMV_MAX_ROWS
        plane = mq.Plane.empty(M, K, self.device, q8=few, op=not few)
        mq.mq_quantize_q8(o.view(M, K), plane)
        y = torch.empty((M, self.hidden), device=self.device)
        return (mq.mq_gemv_q4k if few else mq.mq_gemm_q4k)(plane, self.wo, self.hidden, y)

    def prompt(self, x):
        """The shared prefix: x f32 [T, hidden], its tokens' keys and values become the prefix's rows."""
        T = x.shape[0]
        assert self.prefix_len == 0 and T <= self.prefix.cap
        pos = torch.arange(T, dtype=torch.int32, device=self.device)
        q = self._project(x, pos, self.prefix, pos)
        o = torch.empty((1, T, self.Hq, self.D), device=self.device)
        here = mq.KV(self.prefix.k[:, :T], self.prefix.v[:, :T])
        mq.mq_attn_prefix(q.view(1, T, self.Hq, self.D), None, here,
                          torch.full((1,), T, dtype=torch.int32, device=self.device), o)
        self.shared, self.prefix_len = here, T
        self.position.fill_(T)
        return self._output(o[0])

    def step(self, x):
        """One new token of every sequence: x f32 [batch, hidden]."""
        if self.filled == self.cap:
            self._evict()
        q = self._project(x, self.position, self.own, self.rows + self.length)
        self.length += 1
        self.position += 1
        self.filled += 1
        o = torch.empty((self.batch, 1, self.Hq, self.D), device=self.device)
        mq.mq_attn_prefix(q.view(self.batch, 1, self.Hq, self.D), self.shared if self.prefix_len else None, self.own,
                          self.length, o, score=self.score, score_out=self.score)
        return self._output(o.view(self.batch, self.Hq, self.D))

    def _evict(self):
        mq.mq_kv_evict(self.own, self.length, self.score, self.keep, self.recent, self.spare, self.length,
                       self.spare_score, self.index)
        self.own, self.spare = self.spare, self.own
        self.score, self.spare_score = self.spare_score, self.score
        self.filled = self.keep


def main():
    layer = AttentionLayer(hidden=1024, Hq=8, Hkv=2, D=128, batch=4, prefix_cap=512, cap=64, keep=32, recent=8)
    y = layer.prompt(synth.normal((300, 1024), 1, "prompt", device="cuda"))
    print("prompt:", tuple(y.shape), "norm per row %.3f" % float(y.norm(dim=1).mean()))
    for t in range(100):
        y = layer.step(synth.normal((4, 1024), 2, f"step{t}", device="cuda"))
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    print("100 steps: cache rows", layer.length.tolist(), "positions", layer.position.tolist(),
          "norm per row %.3f" % float(y.norm(dim=1).mean()))


if __name__ == "__main__":
    main()
