"""A key/value cache in 4 bits on pages, measured: head norms and rotation (scaled for long contexts) that fill it
and the rows read back in 16 bits, attention over it, and the page operations of a serving loop (fork, trim, reserve
with copy on write, compaction).

`own` chooses between the plain form (elementary torch operations) and the library's calls.

Rows of a page come in blocks of 16 rows of one head: the keys' 4-bit numbers, the values', the keys' scales, the
values' (one byte per 32 dims). A number is n d with n = nibble - 8 and d = (8 + c % 8) 2^(c / 8 - 18) for a scale byte
c >= 8, c 2^-17 below. The 8 dims 32 b + 8 t + 2 j + h of a key row are nibble j of half h of its 32-bit word
(row, t, b); the dims 32 u + 4 g + i of a value row 8 p + 2 t + c are nibble i of half c of word (p, g, t, u). The value
scales of two neighbouring rows lie side by side.
"""
import math
import random

import torch

own = False

F16, BF16 = "f16", "bf16"
DT = {F16: torch.float16, BF16: torch.bfloat16}
EPS = 1e-6
MOST_CODE = 191          # d = 480


def listed():
    return [
        # one decode step's token: the 14B-shaped layer's heads, contexts four times the trained length
        dict(name="fill_1", op="fill", M=1, n=1, Hq=40, Hkv=8, D=128, rot=128, inter=False, norm=True, factor=4.0, R=64,
             type=F16),
        # the 7B-shaped prompt of 3314 tokens (28 and 4 heads), no scaling
        dict(name="fill_3314", op="fill", M=3314, n=1, Hq=28, Hkv=4, D=128, rot=128, inter=False, norm=True, factor=1.0,
             R=64, type=BF16),
        # three ragged prompts at once, neighbouring pairs, a quarter of each head not rotated, no norm
        dict(name="fill_16384", op="fill", M=16384, n=3, Hq=40, Hkv=8, D=128, rot=96, inter=True, norm=False,
             factor=16.0, R=128, type=F16),
        # one sequence's decode step: latency
        dict(name="decode_1", op="attn", B=1, T=1, Hq=40, Hkv=8, D=128, cap=1000, lo=900, R=64, type=F16),
        # a small server's decode step: 16 ragged sequences, some of them empty, small pages
        dict(name="decode_16", op="attn", B=16, T=1, Hq=28, Hkv=4, D=128, cap=8192, lo=0, R=16, type=BF16),
        # a large one: 64 long sequences
        dict(name="decode_64", op="attn", B=64, T=1, Hq=40, Hkv=8, D=128, cap=20000, lo=9000, R=64, type=F16),
        # five drafted tokens verified at once, narrow heads, odd lengths
        dict(name="verify_4x5", op="attn", B=4, T=5, Hq=28, Hkv=4, D=64, cap=2901, lo=5, R=32, type=BF16),
        # the 7B-shaped prompt's tokens behind 1000 cached ones
        dict(name="prompt_3314", op="attn", B=1, T=3314, Hq=28, Hkv=4, D=128, cap=4314, lo=4314, R=64, type=BF16),
        # beam search of four prompts: every beam continues with one row, four of each, in all 28 layers
        dict(name="next_beams", op="next", n=4, beams=4, rows=1500, trim=0, add=1, layers=28, Hkv=4, D=128, R=64, spare=64),
        # a server's step: 256 sequences drop rejected drafts and reserve five rows each; nothing is shared
        dict(name="next_256", op="next", n=256, beams=1, rows=6000, trim=4, add=5, layers=1, Hkv=8, D=128, R=32, spare=999),
        # a small pool closed up after a few sequences ended
        dict(name="compact_small", op="compact", n=6, rows=700, pages=300, layers=2, Hkv=4, D=64, R=32),
        # a large one: eight layers, half of the pool in use all over it
        dict(name="compact_large", op="compact", n=40, rows=5000, pages=6000, layers=8, Hkv=8, D=128, R=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(28, 4), (40, 8), (32, 8), (16, 16), (12, 1), (64, 8)]


def draw(rng):
    op = rng.choice(["fill", "attn", "attn", "attn", "next", "compact"])
    kind = rng.choice([F16, BF16])
    Hq, Hkv = rng.choice(HEADS)
    R = rng.choice([16, 32, 64, 128, 256])
    if op == "fill":
        D = rng.choice([64, 96, 128, 128, 256])
        M = _log(rng, 1, max(1, 16384 * 56 * 128 // ((Hq + 2 * Hkv) * D)))
        return dict(op=op, M=M, n=min(M, rng.randint(1, 5)), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D - 8]),
                    inter=rng.random() < 0.3, norm=rng.random() < 0.7, factor=rng.choice([1.0, 4.0, 32.0]), R=R, type=kind)
    if op == "attn":
        mode = rng.choice(["decode", "decode", "verify", "prompt"])
        D = rng.choice([64, 128, 128]) if mode == "prompt" else rng.choice([64, 96, 128, 128, 128, 256])
        if mode == "prompt":
            B, T = rng.choice([1, 1, 2, 3]), _log(rng, 40, 3000)
            cap = T + (0 if rng.random() < 0.3 else _log(rng, 1, 4000))
            lo = cap
        else:
            B, T = _log(rng, 1, 64), (rng.randint(2, 8) if mode == "verify" else 1)
            cap = max(T, _log(rng, 8, 20000))
            lo = rng.randint(T, cap)
        while B * cap * Hkv * D > 64 * 20000 * 8 * 128 or B * T * Hq * D * cap > 3314 * 28 * 128 * 4314:
            if B > 1:
                B //= 2
            else:
                T, cap, lo = (T + 1) // 2, (cap + 1) // 2, (lo + 1) // 2
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, cap=cap, lo=lo, R=R, type=kind)
    D, H, layers = rng.choice([64, 128]), rng.choice([1, 4, 8]), rng.choice([1, 3, 8, 28])
    page = layers * R * H * (D + D // 16)
    if op == "next":
        n, beams, add = _log(rng, 1, 128), rng.choice([1, 1, 2, 4]), rng.randint(1, 9)
        rows = _log(rng, 10, 6000)
        while n * (rows // R + 2 + 2 * beams) * page > 6 << 30:
            n, rows = max(1, n // 2), max(10, rows // 2)
        return dict(op=op, n=n, beams=beams, rows=rows, trim=rng.randint(0, 5), add=add, layers=layers, Hkv=H, D=D, R=R,
                    spare=2 * n * beams + rng.randint(0, 500))
    n, rows = _log(rng, 1, 60), _log(rng, 10, 6000)
    while n * (rows // R + 1) * page > 3 << 30:
        n, rows = max(1, n // 2), max(10, rows // 2)
    return dict(op=op, n=n, rows=rows, pages=int(n * (rows // R + 1) * rng.uniform(1.2, 3.0)) + 1, layers=layers, Hkv=H,
                D=D, R=R)


# ------------------------------------------------------------------------------------------- 4-bit rows

def _scale(c):
    """The scales that bytes stand for (64 bits)."""
    c = c.to(torch.int64)
    e, m = c >> 3, (c & 7).double()
    return torch.where(e > 0, torch.ldexp(m + 8.0, e - 18), m * 2.0 ** -17)


def _codes(most):
    """The least code whose 7 d reaches `most` (64 bits), 191 where none does."""
    grid = 7.0 * _scale(torch.arange(MOST_CODE + 1, device=most.device))
    return torch.searchsorted(grid, most.contiguous()).clamp(max=MOST_CODE)


def _rounded(x):
    """Rows [..., D] to (numbers in -7 .. 7, codes [..., D / 32]), in 64 bits."""
    y = x.double().unflatten(-1, (-1, 32))
    c = _codes(y.abs().amax(-1))
    d = _scale(c)[..., None]
    n = torch.where(d > 0, torch.round(y / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(y)).clamp(-7, 7)
    return n, c


def _block_bytes(D):
    return 16 * (D + D // 16)


def _packed(k, v):
    """k, v [P, R, H, D] (numbers and codes) to pages uint8 [P, page bytes]."""
    (kn, kc), (vn, vc) = k, v
    P, R, H, D = kn.shape[0], kn.shape[1], kn.shape[2], vn.shape[-2] * 32
    b = D // 32

    def blocks(t):                                   # [P, H, R / 16, 16, ...]
        return t.transpose(1, 2).unflatten(2, (R // 16, 16))

    ku = blocks((kn + 8).to(torch.uint8).flatten(-2))
    ku = ku.unflatten(-1, (b, 4, 2, 2, 2))           # b, t, j / 2, j % 2, h
    ku = ku.permute(0, 1, 2, 3, 5, 4, 8, 6, 7)       # .., row, t, b, h, j / 2, j % 2
    vu = blocks((vn + 8).to(torch.uint8).flatten(-2)).unflatten(3, (2, 4, 2)).unflatten(-1, (b, 8, 2, 2))
    vu = vu.permute(0, 1, 2, 3, 7, 4, 6, 5, 8, 9)    # .., p, g, t, u, c, i / 2, i % 2
    parts = [(u[..., 0] | (u[..., 1] << 4)).flatten(3) for u in (ku, vu)]
    parts += [blocks(kc.to(torch.uint8)).flatten(3), blocks(vc.to(torch.uint8)).unflatten(3, (8, 2)).transpose(4, 5).flatten(3)]
    return torch.cat(parts, -1).flatten(1)


def _unpacked(pages, R, H, D):
    """uint8 [.., page bytes] to f32 k, v [.., R, H, D]."""
    b, lead = D // 32, pages.shape[:-1]
    x = pages.reshape(-1, H, R // 16, _block_bytes(D))
    n = 8 * D

    def numbers(u):
        return torch.stack([u & 15, u >> 4], -1)

    k = numbers(x[..., :n].unflatten(-1, (16, 4, b, 2, 2))).permute(0, 1, 2, 3, 5, 4, 7, 8, 6).flatten(5)
    v = numbers(x[..., n:2 * n].unflatten(-1, (2, 8, 4, b, 2, 2)))
    v = v.permute(0, 1, 2, 3, 5, 7, 6, 4, 8, 9).flatten(7).flatten(3, 5)          # .., row, u, dims of a block
    k = k.flatten(4).unflatten(-1, (b, 32))
    out = []
    kc, vc = x[..., 2 * n:2 * n + 16 * b].unflatten(-1, (16, b)), x[..., 2 * n + 16 * b:]
    for u, code in ((k, kc), (v, vc.unflatten(-1, (8, b, 2)).transpose(4, 5).flatten(3, 4))):
        d = _scale(code).float()
        y = (u.float() - 8.0) * d[..., None]
        out.append(y.flatten(-2).flatten(2, 3).transpose(1, 2).reshape(*lead, R, H, D))
    return out


# ------------------------------------------------------------------------------------------- inputs

def _normal(g, shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _lens(seed, B, lo, hi):
    r = random.Random(seed)
    return torch.tensor([r.randint(lo, hi) for _ in range(B)], dtype=torch.int32, device="cuda")


def _up(a, b):
    return -(-a // b)


def _freq(rot, factor):
    """Radians per position: base 10^6; for a context `factor` times the trained 32768 the slow pairs turn that much
    slower, the quick ones as they did, those between in proportion."""
    n = rot // 2
    i = torch.arange(n, dtype=torch.float64)
    f = 1e6 ** (-i / n)
    if factor != 1.0:
        turns = 32768 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "fill":
        M, n, Hq, Hkv, D, R, dt = c["M"], c["n"], c["Hq"], c["Hkv"], c["D"], c["R"], DT[c["type"]]
        s["q"] = _normal(g, (M, Hq, D))
        kv = _normal(g, (M, 2 * Hkv, D))             # attn_k and attn_v come out of one product
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["wq"] = _normal(g, (D,), std=0.1).add_(1.0) if c["norm"] else None
        s["wk"] = _normal(g, (D,), std=0.1).add_(1.0) if c["norm"] else None
        s["freq"], s["turn"] = _freq(c["rot"], c["factor"]), float(torch.tensor(0.1 * math.log(c["factor"]) + 1.0))
        base = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        lens = [M // n + (b < M % n) for b in range(n)]
        cap = max(lens)
        s["row"] = torch.cat([torch.arange(x, dtype=torch.int32, device="cuda") for x in lens])
        s["seq"] = torch.repeat_interleave(torch.arange(n, dtype=torch.int32, device="cuda"),
                                           torch.tensor(lens, device="cuda"))
        s["pos"] = s["row"] + base
        s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q_out"] = torch.zeros((M, Hq, D), dtype=dt, device="cuda")
        s["ko"] = torch.zeros((n, cap, Hkv, D), dtype=dt, device="cuda")
        s["vo"] = torch.zeros_like(s["ko"])
        width = _up(cap, R)
        s["table"] = torch.randperm(n * width, generator=g, device="cuda").to(torch.int32).view(n, width)
        s["pages"] = torch.zeros((n * width, R // 16 * Hkv * _block_bytes(D)), dtype=torch.uint8, device="cuda")
        if own:
            from quant_int8_quantized_gb300 import mq
            s["cache"], s["kv"] = mq.KV4(s["pages"], s["table"], R, Hkv, D), mq.KV(s["ko"], s["vo"])
    elif c["op"] == "attn":
        B, T, Hq, Hkv, D, cap, R, dt = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["cap"], c["R"], DT[c["type"]]
        width = _up(cap, R)
        P = B * width
        s["q"] = _normal(g, (B, T, Hq, D), dt, 1.5)
        s["pages"] = torch.empty((P, R // 16 * Hkv * _block_bytes(D)), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (R * Hkv * D))
        for p in range(0, P, step):                  # some 10^8 numbers at once
            m = min(step, P - p)
            s["pages"][p:p + m] = _packed(*(_rounded(_normal(g, (m, R, Hkv, D))) for _ in range(2)))
        s["table"] = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(B, width)
        s["len"] = _lens(seed, B, c["lo"], cap)
        s["out"] = torch.zeros((B, T, Hq, D), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((B, T, Hq), device="cuda")
        if own:
            from quant_int8_quantized_gb300 import mq
            s["cache"] = mq.KV4(s["pages"], s["table"], R, Hkv, D)
            s["ws"] = mq.attn_kv4_workspace(B, T, Hq, Hkv, D, width * R)
    else:
        n, rows, R, H, D, layers = c["n"], c["rows"], c["R"], c["Hkv"], c["D"], c["layers"]
        s["len"] = _lens(seed, n, max(1, rows // 2), rows)
        fork = c["op"] == "next"
        width = _up(rows + (c["add"] if fork else 0), R)
        P = n * width + c["spare"] if fork else max(c["pages"], n * width)
        held = torch.arange(width, device="cuda") < ((s["len"] + R - 1) // R)[:, None]
        place = torch.randperm(P, generator=g, device="cuda")[:n * width].to(torch.int32).view(n, width)
        s["table"] = torch.where(held, place, torch.full_like(place, -1))
        size = R // 16 * H * _block_bytes(D)
        s["pool"] = torch.randint(-2 ** 62, 2 ** 62, (layers, P, size // 8), generator=g, device="cuda")
        m = n * c["beams"] if fork else n
        s["table_out"] = torch.zeros((m, width), dtype=torch.int32, device="cuda")
        s["len_out"] = torch.zeros((m,), dtype=torch.int32, device="cuda")
        s["status"] = torch.zeros((3 if fork else 1,), dtype=torch.int32, device="cuda")
        if fork:
            s["from"] = torch.arange(m, dtype=torch.int32, device="cuda") // c["beams"]
            s["keep"] = (s["len"] - c["trim"])[s["from"].long()].contiguous()
            s["add"] = torch.full((m,), c["add"], dtype=torch.int32, device="cuda")
        else:
            s["where"] = torch.zeros((P,), dtype=torch.int32, device="cuda")
        if own:
            from quant_int8_quantized_gb300 import mq
            s["pages"] = mq.Pool(s["pool"].view(torch.uint8), R)
            s["ws"] = mq.pages_workspace(s["pages"], m, width)
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    return {"fill": _fill, "attn": _attn, "next": _next, "compact": _compact}[s["case"]["op"]](s)


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


def _fill(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_qk_norm_rope_kv4(s["q"], s["k"], s["v"], s["q_out"], s["cache"], s["seq"], s["row"], s["pos"], s["freq"],
                               wq=s["wq"], wk=s["wk"], eps=EPS, interleaved=c["inter"], rot_scale=s["turn"])
        mq.mq_kv4_read(s["cache"], s["len"], s["kv"])
    else:
        # angles, and keys and values next to a border between two of the 15 numbers, want 64 bits
        n, dt = c["rot"] // 2, DT[c["type"]]
        t = s["pos"].double()[:, None] * s["freq"].double()
        cos, sin = (t.cos() * s["turn"])[:, None], (t.sin() * s["turn"])[:, None]
        s["q_out"].copy_(_rotate(s["q"], s["wq"], cos.float(), sin.float(), n, c["inter"]))
        k = _rotate(s["k"].double(), None if s["wk"] is None else s["wk"].double(), cos, sin, n, c["inter"])
        for x, out in ((k, "ko"), (s["v"], "vo")):
            m, code = _rounded(x)
            s[out][s["seq"].long(), s["row"].long()] = (m * _scale(code)[..., None]).flatten(-2).to(dt)
    return {"q": s["q_out"], "k": s["ko"], "v": s["vo"]}


def _attn(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_attn_kv4(s["q"], s["cache"], s["len"], s["out"], lse=s["lse"], ws=s["ws"])
        return [s["out"], s["lse"]]
    B, T, Hq, Hkv, D, R = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["R"]
    G = Hq // Hkv
    k, v = (x.flatten(1, 2) for x in _unpacked(s["pages"][s["table"].long()], R, Hkv, D))       # [B, rows, Hkv, D]
    j, t = torch.arange(k.shape[1], device="cuda"), torch.arange(T, device="cuda")
    q = (s["q"].float() / math.sqrt(D)).view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, T, G, -1)
    seen = j < (s["len"][:, None] - T + 1 + t)[:, :, None]                                      # [B, T, rows]
    x = x.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    m = x.amax(-1)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)                                 # a row that sees nothing
    x = (x - m[..., None]).exp()
    total = x.sum(-1)
    inv = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    o = (x.view(B, Hkv, T * G, -1) @ v.permute(0, 2, 1, 3)).view(B, Hkv, T, G, D) * inv[..., None]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D))
    s["lse"].copy_((m + total.log()).permute(0, 2, 1, 3).reshape(B, T, Hq))
    return [s["out"], s["lse"]]


def _next(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_pages_next(s["pages"], s["table"], s["len"], s["table_out"], s["len_out"], s["status"], frm=s["from"],
                         keep=s["keep"], add=s["add"], ws=s["ws"])
        return {"table": s["table_out"], "len": s["len_out"], "status": s["status"], "pool": s["pool"]}
    R, P, width = c["R"], s["pool"].shape[1], s["table"].shape[1]
    old = s["from"].long()
    m = len(old)
    L = torch.minimum(s["len"][old], s["keep"]).clamp(min=0).long()
    kept, i = (L + R - 1) // R, torch.arange(width, device="cuda")
    table = s["table"][old].long()
    table = torch.where(i < kept[:, None], table, torch.full_like(table, -1))
    held = torch.bincount(table.flatten() + 1, minlength=P + 1)[1:]
    long = L + s["add"] > width * R
    add = torch.where(long, torch.zeros_like(L), s["add"].clamp(min=0).long())
    last = table.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0]
    part = (add > 0) & (L % R != 0) & (last >= 0)                     # goes on in the page of its last row
    page = torch.where(part, last, torch.full_like(last, P))
    b = torch.arange(m, device="cuda")
    writers = torch.bincount(page, minlength=P + 1)
    first = torch.full((P + 1,), m, device="cuda").scatter_reduce_(0, page, b, "amin")
    held = torch.cat([held, held.new_zeros(1)])
    copy = part & (held[page] > 1) & ~((writers[page] == held[page]) & (first[page] == b))
    fresh = (L + add + R - 1) // R - kept
    want = fresh + copy
    free = torch.where(held[:P] == 0, torch.arange(P, device="cuda"), torch.full((P,), P, device="cuda")).sort().values
    n_free, total = (held[:P] == 0).sum(), want.sum()
    enough = total <= n_free
    rank = (want.cumsum(0) - want)[:, None] + i - (kept - copy.long())[:, None]
    new = (i >= (kept - copy.long())[:, None]) & (i < (kept + fresh)[:, None]) & enough
    s["table_out"].copy_(torch.where(new, free[rank.clamp(0, P - 1)], table))
    s["len_out"].copy_(L + add * enough)
    s["status"].copy_(torch.stack([(total - n_free).clamp(min=0), n_free - total * enough, long.sum()]))
    src = last[copy & enough]
    dst = s["table_out"].long().gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0][copy & enough]
    s["pool"][:, dst] = s["pool"][:, src]
    return {"table": s["table_out"], "len": s["len_out"], "status": s["status"], "pool": s["pool"]}


def _compact(s):
    c = s["case"]
    if own:
        from quant_int8_quantized_gb300 import mq
        mq.mq_pages_compact(s["pages"], s["table"], s["len"], s["table_out"], s["where"], s["status"], ws=s["ws"])
        return {"table": s["table_out"], "where": s["where"], "live": s["status"], "pool": s["pool"]}
    R, P, width = c["R"], s["pool"].shape[1], s["table"].shape[1]
    inside = torch.arange(width, device="cuda") < ((s["len"] + R - 1) // R)[:, None]
    page = torch.where(inside & (s["table"] >= 0), s["table"], torch.full_like(s["table"], P)).long()
    live = torch.zeros((P + 1,), dtype=torch.bool, device="cuda").scatter_(0, page.flatten(), True)[:P]
    n, p = live.sum(), torch.arange(P, device="cuda")
    src, dst = (live & (p >= n)).nonzero()[:, 0], (~live & (p < n)).nonzero()[:, 0]
    where = torch.where(live, p, torch.full_like(p, -1))
    where[src] = dst
    s["where"].copy_(where)
    s["table_out"].copy_(torch.cat([where, where.new_full((1,), -1)])[page])
    s["status"].copy_(n[None])
    s["pool"][:, dst] = s["pool"][:, src]
    return {"table": s["table_out"], "where": s["where"], "live": s["status"], "pool": s["pool"]}


# ------------------------------------------------------------------------------------------- the least work

def work(case):
    c = case
    if c["op"] == "fill":
        n, kv = c["M"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"], c["M"] * 2 * c["Hkv"] * c["D"]
        return {"bytes": 4 * n + 2 * (n - kv) + kv * (17 / 32 + 17 / 32 + 2), "flops": 10 * n}
    if c["op"] == "attn":
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        n = (c["lo"] + c["cap"]) / 2
        return {"bytes": 4 * B * T * Hq * D + 4 * B * T * Hq + 2 * B * n * Hkv * D * 17 / 32,
                "flops": 4 * D * B * T * Hq * (n - (T - 1) / 2)}
    page = c["layers"] * c["R"] * c["Hkv"] * (c["D"] + c["D"] // 16)
    width = _up(c["rows"] + c.get("add", 0), c["R"])
    if c["op"] == "next":       # of the beams of a prompt one goes on in the page that they share
        copies = c["n"] * (c["beams"] - 1) * (1 - 1 / c["R"])
        return {"bytes": 4 * c["n"] * (1 + c["beams"]) * width + 2 * copies * page, "flops": 0}
    held = c["n"] * (0.75 * c["rows"] / c["R"] + 0.5)
    moved = held * (1 - min(1, held / max(c["pages"], c["n"] * width)))
    return {"bytes": 8 * c["n"] * width + 4 * c["pages"] + 2 * moved * page, "flops": 0}


# ------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    global own
    if case["op"] not in ("fill", "attn"):
        return None             # whole numbers and bytes that move
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return (_exact_fill if case["op"] == "fill" else _exact_attn)(s)


def _levels(x):
    """x [rows, D] in 64 bits as the nearest n d, block by block."""
    out = torch.zeros_like(x)
    scales = [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 24) for m in range(8)]
    scales = torch.tensor(scales, dtype=torch.float64, device=x.device)
    for b in range(0, x.shape[1], 32):
        y = x[:, b:b + 32]
        need = y.abs().max(1).values / 7
        d = scales[(scales[None, :] * 7 < need[:, None] * 7).sum(1).clamp(max=len(scales) - 1)][:, None]
        out[:, b:b + 32] = torch.where(d > 0, torch.round(y / d.clamp(min=2.0 ** -20)).clamp(-7, 7) * d, 0.0)
    return out


def _exact_fill(s):
    c = s["case"]
    n, D = c["rot"] // 2, c["D"]
    angle = s["pos"].double()[:, None] * s["freq"].double()[None]
    turn = torch.polar(torch.full_like(angle, s["turn"]), angle)[:, None]

    def of(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x.square().sum(-1, keepdim=True) / D) + EPS).sqrt() * w.double()
        y = x.clone()
        first = slice(0, 2 * n, 2) if c["inter"] else slice(0, n)
        second = slice(1, 2 * n, 2) if c["inter"] else slice(n, 2 * n)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": of(s["q"], s["wq"])}
    for name, x in (("k", of(s["k"], s["wk"])), ("v", s["v"].double())):
        y = torch.zeros(s["ko"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for b, m in enumerate(s["len"].tolist()):
            y[b, :m] = torch.stack([_levels(x[at:at + m, h]) for h in range(c["Hkv"])], 1)
            at += m
        out[name] = y
    return out


def _exact_attn(s):
    c = s["case"]
    B, T, Hq, Hkv, D, R = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["R"]
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    lens = s["len"].tolist()
    # where dim d of row r of a block lies: byte and shift, of keys and of values
    r, d = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    b, t, j, h = d // 32, d % 32 // 8, d % 8 // 2, d % 2
    kb, ks = (r * 4 * (D // 32) + t * (D // 32) + b) * 4 + 2 * h + j // 2, 4 * (j % 2)
    g, i = d % 32 // 4, d % 4
    vb = 8 * D + (((r // 8 * 8 + g) * 4 + r % 8 // 2) * (D // 32) + b) * 4 + 2 * (r % 2) + i // 2
    vs = 4 * (i % 2)
    kc = 16 * D + r * (D // 32) + b
    vc = 16 * D + 16 * (D // 32) + (r // 2 * (D // 32) + b) * 2 + r % 2
    scales = [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 32) for m in range(8)]
    scales = torch.tensor(scales, dtype=torch.float64, device="cuda")
    for q in range(B):
        n = lens[q]
        if n == 0:
            continue
        pages = s["pages"][s["table"][q, :_up(n, R)].long()].view(-1, Hkv, R // 16, _block_bytes(D))
        for hk in range(Hkv):
            x = pages[:, hk].reshape(-1, _block_bytes(D))                       # blocks of 16 rows, in order
            keys = (((x[:, kb] >> ks) & 15).double() - 8) * scales[x[:, kc].long()]
            vals = (((x[:, vb] >> vs) & 15).double() - 8) * scales[x[:, vc].long()]
            keys, vals = keys.view(-1, D)[:n], vals.view(-1, D)[:n]
            z = s["q"][q, :, hk * G:(hk + 1) * G].double().transpose(0, 1) @ keys.T / D ** 0.5     # [G, T, n]
            if T > 1:                                                          # the last T keys are the queries' own
                late = torch.ones((T, n), dtype=torch.bool, device="cuda").triu_(n - T + 1)
                z.masked_fill_(late, float("-inf"))
            l = torch.logsumexp(z, -1)
            p = torch.nan_to_num((z - l[..., None]).exp_(), nan=0.0)
            out[q, :, hk * G:(hk + 1) * G] = (p @ vals).transpose(0, 1)
            lse[q, :, hk * G:(hk + 1) * G] = l.T
    return [out, lse]
