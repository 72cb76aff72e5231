"""What lies between a decoder layer's attn_q|k|v and attn_o products, measured: the per-head norms and
rotation that fill a key/value cache, attention over a shared prefix and each sequence's own cache, and
the eviction of a cache's least attended keys.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math
import random

import torch

own = False

F16, BF16 = "f16", "bf16"
DT = {F16: torch.float16, BF16: torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one new token of one sequence: the 14B-shaped decode step's heads, 40 query and 8 key heads
        dict(name="rope_decode_1", op="rope", M=1, Hq=40, Hkv=8, D=128, rot=128, axes=1, inter=False, norm=True,
             cap=16, type=F16),
        # the 7B-shaped prompt of 3314 tokens (28 and 4 heads), an image's three axes of positions
        dict(name="rope_prefill_3314", op="rope", M=3314, Hq=28, Hkv=4, D=128, rot=128, axes=3, inter=False, norm=True,
             cap=1, type=BF16),
        # a long prompt, neighbouring pairs, a quarter of each head left as it is, no norm
        dict(name="rope_prefill_16384", op="rope", M=16384, Hq=40, Hkv=8, D=128, rot=96, axes=1, inter=True,
             norm=False, cap=1, type=F16),
        # one sequence's decode step after a short system prompt: latency
        dict(name="attn_decode_1", op="attn", B=1, T=1, Hq=40, Hkv=8, D=128, P=512, cap=64, lo=1, scores=False,
             type=F16),
        # a small server's decode step: 16 ragged sequences on a 4k system prompt
        dict(name="attn_decode_16", op="attn", B=16, T=1, Hq=28, Hkv=4, D=128, P=4096, cap=1000, lo=0, scores=False,
             type=BF16),
        # a large one: 64 sequences on a long shared document
        dict(name="attn_decode_64", op="attn", B=64, T=1, Hq=40, Hkv=8, D=128, P=32768, cap=2048, lo=17, scores=False,
             type=F16),
        # a decode step that keeps the books for eviction, nothing shared
        dict(name="attn_scores_8", op="attn", B=8, T=1, Hq=40, Hkv=8, D=128, P=0, cap=4096, lo=4000, scores=True,
             type=BF16),
        # five drafted tokens verified at once, narrow heads, odd lengths
        dict(name="attn_verify_4x5", op="attn", B=4, T=5, Hq=28, Hkv=4, D=64, P=2049, cap=777, lo=5, scores=False,
             type=F16),
        # the 7B-shaped prompt: causal attention of 3314 tokens behind a shared prefix of 1000
        dict(name="attn_prefill_3314", op="attn", B=1, T=3314, Hq=28, Hkv=4, D=128, P=1000, cap=3314, lo=3314,
             scores=False, type=BF16),
        # one sequence's small cache cut to half
        dict(name="evict_1", op="evict", B=1, H=8, D=128, cap=512, lo=512, keep=256, recent=32, type=F16),
        # a batch of ragged caches cut to a quarter
        dict(name="evict_32", op="evict", B=32, H=8, D=128, cap=4096, lo=900, keep=1024, recent=128, type=BF16),
        # two very long caches cut to an eighth
        dict(name="evict_2x131072", op="evict", B=2, H=4, D=128, cap=131072, lo=131000, keep=16384, recent=1001,
             type=F16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(28, 4), (40, 8), (32, 8), (16, 16), (12, 1), (64, 8)]


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "attn", "evict"])
    kind = rng.choice([F16, BF16])
    Hq, Hkv = rng.choice(HEADS)
    if op == "rope":
        D = rng.choice([64, 96, 128, 128, 256])
        M = _log(rng, 1, max(1, 16384 * 56 * 128 // ((Hq + 2 * Hkv) * D)))
        rot = rng.choice([D, D, D // 2, D - 8])
        return dict(op=op, M=M, Hq=Hq, Hkv=Hkv, D=D, rot=rot, axes=rng.choice([1, 1, 3]), inter=rng.random() < 0.3,
                    norm=rng.random() < 0.7, cap=rng.choice([1, 3]), type=kind)
    if op == "attn":
        D = rng.choice([64, 128, 128])
        mode = rng.choice(["decode", "decode", "scores", "verify", "prompt"])
        P = 0 if rng.random() < 0.2 else _log(rng, 16, 32768)
        if mode == "prompt":
            B, T = rng.choice([1, 1, 2, 3]), _log(rng, 40, 3000)
            P = min(P, 4096)
            cap = T + (0 if rng.random() < 0.5 else _log(rng, 1, 1000))
        else:
            B, T = _log(rng, 1, 64), (rng.randint(2, 8) if mode == "verify" else 1)
            cap = _log(rng, 8, 4096)
        cap = max(cap, T)
        lo = cap if mode == "prompt" else rng.randint(T, cap)
        most = 64 * 40 * 128 * 34816     # the listed decode step of 64 sequences
        while B * T * Hq * D * (P + cap) > most:
            if P > cap:
                P //= 2
            elif B > 1:
                B //= 2
            else:
                T, cap, lo = T // 2, cap // 2, lo // 2
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, cap=cap, lo=lo, scores=mode == "scores", type=kind)
    D, H = rng.choice([64, 128]), rng.choice([1, 4, 8])
    cap = _log(rng, 64, 131072)
    B = _log(rng, 1, max(1, min(32, 2 * 4 * 131072 // (H * cap))))
    keep = max(2, int(cap * rng.uniform(0.05, 0.9)))
    return dict(op=op, B=B, H=H, D=D, cap=cap, lo=rng.randint(0, cap), keep=keep, recent=rng.randint(0, keep // 2),
                type=kind)


# ------------------------------------------------------------------------------------------- inputs

def _normal(g, shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _lens(seed, B, lo, hi):
    r = random.Random(seed)
    return torch.tensor([r.randint(lo, hi) for _ in range(B)], dtype=torch.int32, device="cuda")


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).to(torch.float32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    c, dt = dict(case), DT[case["type"]]
    s = {"case": c}
    if c["op"] == "rope":
        M, Hq, Hkv, D = c["M"], c["Hq"], c["Hkv"], c["D"]
        n = c["rot"] // 2
        s["q"] = _normal(g, (M, Hq, D))
        kv = _normal(g, (M, 2 * Hkv, D))          # attn_k and attn_v come out of one product
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["wq"] = _normal(g, (D,), std=0.1).add_(1.0) if c["norm"] else None
        s["wk"] = _normal(g, (D,), std=0.1).add_(1.0) if c["norm"] else None
        s["freq"] = _inv_freq(c["rot"])
        m = torch.arange(M, dtype=torch.int32, device="cuda")
        base = int(torch.randint(0, 8192, (1,), generator=g, device="cuda"))
        if c["axes"] == 1:
            s["pos"], s["axis"] = (m + base).view(1, M), None
        else:                                     # frames of 32 x 24 patches
            s["pos"] = torch.stack([m // 768 + base, m // 32 % 24 + base, m % 32 + base]).contiguous()
            a = n // 4
            s["axis"] = torch.tensor([0] * a + [1] * ((n - a) // 2) + [2] * (n - a - (n - a) // 2), dtype=torch.uint8,
                                     device="cuda")
        s["q_out"] = torch.zeros((M, Hq, D), dtype=dt, device="cuda")
        s["kc"] = torch.zeros((M, c["cap"], Hkv, D), dtype=dt, device="cuda")   # M caches of `cap` rows
        s["vc"] = torch.zeros_like(s["kc"])
        s["slot"] = m * c["cap"] + torch.randint(0, c["cap"], (M,), generator=g, device="cuda", dtype=torch.int32)
        if own:
            from quant_int8_quantized_gb300 import mq
            s["kv"] = mq.KV(s["kc"], s["vc"])
    elif c["op"] == "attn":
        B, T, Hq, Hkv, D, P, cap = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["P"], c["cap"]
        s["q"] = _normal(g, (B, T, Hq, D), dt, 1.5)
        s["pk"], s["pv"] = _normal(g, (1, P, Hkv, D), dt), _normal(g, (1, P, Hkv, D), dt)
        s["k"], s["v"] = _normal(g, (B, cap, Hkv, D), dt), _normal(g, (B, cap, Hkv, D), dt)
        s["len"] = _lens(seed, B, c["lo"], cap)
        s["score"] = torch.rand((B, Hkv, cap), generator=g, device="cuda") if c["scores"] else None
        s["out"] = torch.zeros((B, T, Hq, D), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((B, T, Hq), device="cuda")
        s["score_out"] = torch.zeros((B, Hkv, cap), device="cuda") if c["scores"] else None
        if own:
            from quant_int8_quantized_gb300 import mq
            s["prefix"] = mq.KV(s["pk"], s["pv"]) if P else None
            s["cache"] = mq.KV(s["k"], s["v"])
            s["ws"] = mq.attn_workspace(B, T, Hq, Hkv, D, P, cap, scores=c["scores"])
    else:
        B, H, D, cap, keep = c["B"], c["H"], c["D"], c["cap"], c["keep"]
        s["k"], s["v"] = _normal(g, (B, cap, H, D), dt), _normal(g, (B, cap, H, D), dt)
        # accumulated weights: skewed, many keys with next to none
        s["score"] = torch.rand((B, H, cap), generator=g, device="cuda").pow_(6.0)
        s["len"] = _lens(seed, B, c["lo"], cap)
        s["dk"] = torch.zeros((B, keep, H, D), dtype=dt, device="cuda")
        s["dv"] = torch.zeros_like(s["dk"])
        s["dscore"] = torch.zeros((B, H, keep), device="cuda")
        s["dlen"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
        s["index"] = torch.zeros((B, H, keep), dtype=torch.int32, device="cuda")
        if own:
            from quant_int8_quantized_gb300 import mq
            s["src"], s["dst"] = mq.KV(s["k"], s["v"]), mq.KV(s["dk"], s["dv"])
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    return {"rope": _rope, "attn": _attn, "evict": _evict}[s["case"]["op"]](s)


def _rotate(x, w, cos, sin, n, inter):
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if inter:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, x[..., 2 * n:]], -1)


def _rope(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_qk_norm_rope(s["q"], s["k"], s["v"], s["q_out"], s["kv"], s["slot"], s["pos"], s["freq"], axis=s["axis"],
                           wq=s["wq"], wk=s["wk"], eps=EPS, interleaved=c["inter"])
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    pos = s["pos"].float()
    pos = pos[0][:, None] if s["axis"] is None else pos[s["axis"].long()].T     # [M, n]
    t = pos * s["freq"]
    cos, sin, n, dt = t.cos()[:, None], t.sin()[:, None], c["rot"] // 2, DT[c["type"]]
    s["q_out"].copy_(_rotate(s["q"], s["wq"], cos, sin, n, c["inter"]))
    at = s["slot"].long()
    s["kc"].view(-1, c["Hkv"], c["D"])[at] = _rotate(s["k"], s["wk"], cos, sin, n, c["inter"]).to(dt)
    s["vc"].view(-1, c["Hkv"], c["D"])[at] = s["v"].to(dt)
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _attn(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_attn_prefix(s["q"], s["prefix"], s["cache"], s["len"], s["out"], lse=s["lse"], score=s["score"],
                          score_out=s["score_out"], ws=s["ws"])
        return [s[k] for k in ("out", "lse", "score_out") if s[k] is not None]
    B, T, Hq, Hkv, D, P, cap = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["P"], c["cap"]
    G = Hq // Hkv
    q = s["q"].float().view(B, T, Hkv, G, D) / math.sqrt(D)
    qo = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    so = (qo @ s["k"].float().permute(0, 2, 3, 1)).view(B, Hkv, T, G, cap)
    j, t = torch.arange(cap, device="cuda"), torch.arange(T, device="cuda")
    seen = j < (s["len"][:, None] - T + 1 + t)[:, :, None]                       # [B, T, cap]
    so = so.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    qp = q.permute(2, 0, 1, 3, 4).reshape(Hkv, B * T * G, D)
    sp = qp @ s["pk"][0].float().permute(1, 2, 0)                                # [Hkv, B T G, P]
    sp = sp.view(Hkv, B, T, G, P).permute(1, 0, 2, 3, 4)                         # [B, Hkv, T, G, P]
    m = so.amax(-1)
    if P:
        m = torch.maximum(m, sp.amax(-1))
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)                  # a row that sees nothing
    so, sp = (so - m[..., None]).exp(), (sp - m[..., None]).exp()
    total = so.sum(-1) + sp.sum(-1)
    inv = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    o = (so.view(B, Hkv, T * G, cap) @ s["v"].float().permute(0, 2, 1, 3)).view(B, Hkv, T, G, D)
    op = sp.permute(1, 0, 2, 3, 4).reshape(Hkv, B * T * G, P) @ s["pv"][0].float().permute(1, 0, 2)
    o = (o + op.view(Hkv, B, T, G, D).permute(1, 0, 2, 3, 4)) * inv[..., None]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D))
    s["lse"].copy_((m + total.log()).permute(0, 2, 1, 3).reshape(B, T, Hq))
    if c["scores"]:
        w = s["score"] + (so * inv[..., None]).sum((2, 3))
        s["score_out"].copy_(torch.where((j < s["len"][:, None])[:, None], w, torch.zeros_like(w)))
    return [s[k] for k in ("out", "lse", "score_out") if s[k] is not None]


def _evict(s):
    c = s["case"]
    B, H, D, cap, keep, recent = c["B"], c["H"], c["D"], c["cap"], c["keep"], c["recent"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_kv_evict(s["src"], s["len"], s["score"], keep, recent, s["dst"], s["dlen"], s["dscore"], s["index"])
    else:
        n, j = s["len"].long(), torch.arange(cap, device="cuda")
        inside = (j < n[:, None])[:, None].expand(B, H, cap)
        last = (j >= (n - recent)[:, None])[:, None]
        rank = torch.where(last, torch.full_like(s["score"], float("inf")), s["score"])
        rank = torch.where(inside, rank, torch.full_like(rank, float("-inf")))
        best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
        kept = torch.zeros((B, H, cap), dtype=torch.bool, device="cuda").scatter_(-1, best, True) & inside
        place = torch.where(kept, j, torch.full_like(j, cap)).sort(dim=-1).values[..., :keep]
        there = place < cap
        at = place.clamp(max=cap - 1)
        s["index"].copy_(torch.where(there, place, torch.full_like(place, -1)))
        s["dscore"].copy_(s["score"].gather(-1, at) * there)
        rows = at.permute(0, 2, 1)[..., None].expand(B, keep, H, D)
        for src, dst in (("k", "dk"), ("v", "dv")):
            s[dst].copy_(s[src].gather(1, rows) * there.permute(0, 2, 1)[..., None])
        s["dlen"].copy_(n.clamp(max=keep))
    return {"k": s["dk"], "v": s["dv"], "score": s["dscore"], "len": s["dlen"], "index": s["index"]}


# ------------------------------------------------------------------------------------------- the least work

def work(case):
    c = case
    if c["op"] == "rope":
        n = c["M"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 6 * n, "flops": 10 * n}
    if c["op"] == "attn":
        B, T, Hq, Hkv, D, P = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["P"]
        n = (c["lo"] + c["cap"]) / 2
        b = 4 * B * T * Hq * D + 4 * B * T * Hq + 4 * Hkv * D * (P + B * n) + (8 * B * Hkv * n if c["scores"] else 0)
        return {"bytes": b, "flops": 4 * D * B * T * Hq * (P + n - (T - 1) / 2)}
    B, H, D, cap, keep = c["B"], c["H"], c["D"], c["cap"], c["keep"]
    n = (c["lo"] + cap) / 2
    k = min(keep, n)
    return {"bytes": B * H * (4 * n + k * (2 * 2 * 2 * D + 8)), "flops": B * H * n}


# ------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    n, axes = c["rot"] // 2, s["axis"]
    axes = torch.zeros(n, dtype=torch.long, device="cuda") if axes is None else axes.long()
    angle = s["pos"].double().index_select(0, axes).mul(s["freq"].double()[:, None]).T.contiguous()   # [M, n]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def of(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x.square().sum(-1, keepdim=True) / c["D"]) + EPS).sqrt() * w.double()
        y = x.clone()
        first = slice(0, 2 * n, 2) if c["inter"] else slice(0, n)
        second = slice(1, 2 * n, 2) if c["inter"] else slice(n, 2 * n)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k = torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    m, slot = torch.arange(c["M"], device="cuda"), s["slot"].long()
    k[m, slot % c["cap"]] = of(s["k"], s["wk"])
    v[m, slot % c["cap"]] = s["v"].double()
    return {"q": of(s["q"], s["wq"]), "k": k, "v": v}


def _exact_attn(s):
    c = s["case"]
    B, T, Hq, Hkv, D, cap = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["cap"]
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    score = torch.zeros((B, Hkv, cap), dtype=torch.float64, device="cuda")
    lens = s["len"].tolist()
    for h in range(Hkv):
        pk, pv = s["pk"][0, :, h].double(), s["pv"][0, :, h].double()
        for b in range(B):
            n = lens[b]
            keys = torch.cat([pk, s["k"][b, :n, h].double()])
            vals = torch.cat([pv, s["v"][b, :n, h].double()])
            if not len(keys):
                continue
            q = s["q"][b, :, h * G:(h + 1) * G].double().transpose(0, 1)        # [G, T, D]
            z = q @ keys.T / D ** 0.5
            if T > 1:                                                          # the last T keys are the queries' own
                late = torch.ones((T, len(keys)), dtype=torch.bool, device="cuda").triu_(len(keys) - T + 1)
                z.masked_fill_(late, float("-inf"))
            l = torch.logsumexp(z, -1)
            p = (z - l[..., None]).exp_()
            out[b, :, h * G:(h + 1) * G] = (p @ vals).transpose(0, 1)
            lse[b, :, h * G:(h + 1) * G] = l.T
            if c["scores"]:
                score[b, h, :n] = s["score"][b, h, :n].double() + p.sum((0, 1))[len(pk):]
    return [out, lse] + ([score] if c["scores"] else [])


def _exact_evict(s):
    c = s["case"]
    B, H, D, keep, recent = c["B"], c["H"], c["D"], c["keep"], c["recent"]
    k = torch.zeros((B, keep, H, D), dtype=torch.float64, device="cuda")
    v, score = torch.zeros_like(k), torch.zeros((B, H, keep), dtype=torch.float64, device="cuda")
    index = torch.full((B, H, keep), -1, dtype=torch.int32, device="cuda")
    lens = s["len"].tolist()
    for b in range(B):
        n = lens[b]
        for h in range(H):
            if n <= keep:
                take = list(range(n))
            else:
                x = s["score"][b, h, :n - recent].tolist()
                take = sorted(sorted(range(n - recent), key=lambda i: (-x[i], i))[:keep - recent])
                take += list(range(n - recent, n))
            t = torch.tensor(take, dtype=torch.long, device="cuda")
            m = len(take)
            k[b, :m, h], v[b, :m, h] = s["k"][b, t, h].double(), s["v"][b, t, h].double()
            score[b, h, :m], index[b, h, :m] = s["score"][b, h, t].double(), t.int()
    return {"k": k, "v": v, "score": score, "len": torch.clamp(s["len"], max=keep), "index": index}
