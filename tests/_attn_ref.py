"""Plain 64-bit forms of the calls between attn_q|k|v and attn_o, for the GPU tests, with error
bounds that follow from the arithmetic include/mq.h states. Written from the definitions, one
sequence and head at a time, on whatever device the inputs are."""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # unit roundoff
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def attention(q, pk, pv, k, v, lens, scale, out_dtype, score=None, only=None):
    """(out, lse, score_out) and their bounds, f64. q [B, T, Hq, D]; pk, pv [P, Hkv, D] or None; k, v
    [B, cap, Hkv, D] or None; lens: list. Only visible keys are ever touched. only: the queries looked at, by
    number (the others' entries mean nothing).

    Bounds: the products q.k are f32 sums of exact products, off by at most 2^-20 sum |q k| scale here
    (D <= 256 terms), the exponentials by 2^-20 relative (exp2 and the f32 rounding of its argument
    among it), so each weight by e relative; the weights are rounded to the caches' type for the second product
    (u relative, or half the smallest subnormal against a maximum of 1, so against a sum of at
    least 1), whose f32 sums add 2^-16 of sum p |v| at most; the output is rounded once."""
    B, T, Hq, D = q.shape
    Hkv = (k if k is not None else pk).shape[-2]
    G, dev, dt = Hq // Hkv, q.device, q.dtype
    cap = 0 if k is None else k.shape[1]
    f64 = dict(dtype=torch.float64, device=dev)
    out, b_out = torch.zeros((B, T, Hq, D), **f64), torch.zeros((B, T, Hq, D), **f64)
    lse, b_lse = torch.full((B, T, Hq), -float("inf"), **f64), torch.zeros((B, T, Hq), **f64)
    sc, b_sc = torch.zeros((B, Hkv, cap), **f64), torch.zeros((B, Hkv, cap), **f64)
    for b in range(B):
        n = 0 if k is None else min(max(int(lens[b]), 0), cap)
        for h in range(Hq):
            hk = h // G
            for t in (range(T) if only is None else only):
                own = max(0, n - T + 1 + t)
                ks, vs = [], []
                if pk is not None:
                    ks.append(pk[:, hk].double())
                    vs.append(pv[:, hk].double())
                if own:
                    ks.append(k[b, :own, hk].double())
                    vs.append(v[b, :own, hk].double())
                if not ks or sum(len(x) for x in ks) == 0:
                    continue
                K, V, x = torch.cat(ks), torch.cat(vs), q[b, t, h].double()
                s = K @ x * scale
                e = 2.0 ** -20 * float((K.abs() @ x.abs()).max() * abs(scale)) + 2.0 ** -20
                l = torch.logsumexp(s, 0)
                p = (s - l).exp()
                o, A = p @ V, p @ V.abs()
                out[b, t, h], lse[b, t, h] = o, l
                b_out[b, t, h] = (A * (U[dt] + 3 * e + 2.0 ** -16) + TINY[dt] * V.abs().sum(0)) * 1.01 + \
                    U[out_dtype] * o.abs() * 1.01 + TINY[out_dtype]
                b_lse[b, t, h] = 2 * e + 2.0 ** -21 * (1 + l.abs())
                if score is not None and own:
                    w = p[len(p) - own:]
                    sc[b, hk, :own] += w
                    b_sc[b, hk, :own] += w * (3 * e + 2.0 ** -19)
        if score is not None:
            for hk in range(Hkv):
                b_sc[b, hk, :n] += 2.0 ** -21 * (score[b, hk, :n].double().abs() + sc[b, hk, :n])
                sc[b, hk, :n] += score[b, hk, :n].double()
    return (out, lse, sc), (b_out, b_lse, b_sc)


def rope(x, w, eps, pos, freq, axis, n_axes, interleaved, dtype):
    """(y, bound): per-head norm (w None: none) and rotation of x f32 [M, H, D]; pos [n_axes, M]."""
    M, H, D = x.shape
    y = x.double()
    if w is not None:
        y = y * w.double() / ((y * y).mean(-1, keepdim=True) + eps).sqrt()
    n = 0 if freq is None else freq.numel()
    normed = y.clone()
    if n:
        ax = [0] * n if axis is None else [min(int(a), n_axes - 1) for a in axis]
        for i in range(n):
            ang = pos[ax[i]].double() * freq[i].double()
            c, s = ang.cos()[:, None], ang.sin()[:, None]
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            a, b = normed[..., ia], normed[..., ib]
            y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    # f32: the norm's factor, two products and a sum, the angle in turns rounded to f32 (2^-24 of half a turn
    # at most: pi 2^-24 rad) and sincospi: within 2^-20 of the pair's size; then one rounding
    if n:
        size = torch.zeros_like(y)
        for i in range(n):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            r = (normed[..., ia].square() + normed[..., ib].square()).sqrt()
            size[..., ia] = size[..., ib] = r
        size[..., 2 * n:] = normed[..., 2 * n:].abs()
    else:
        size = normed.abs()
    return y, size * 2.0 ** -20 + U[dtype] * y.abs() * 1.01 + TINY[dtype]


def evict(score, length, keep, recent):
    """Kept rows of one head, in order: score a list of floats, NaN the lowest, ties to the lower row."""
    if length <= keep:
        return list(range(length))
    cand = length - recent
    low = lambda x: (1, 0.0) if x != x else (0, -x)   # noqa: E731
    best = sorted(range(cand), key=lambda i: (low(score[i]), i))[:keep - recent]
    return sorted(best) + list(range(cand, length))
