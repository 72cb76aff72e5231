"""Plain forms of the calls on 4-bit caches and pages, for the tests, written from include/mq.h."""
import torch

from quant_int8_quantized_gb300 import mq

SCALES = [c * 2.0 ** -17 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 18) for c in range(256)]
MOST = 191


def block_bytes(D):
    return 17 * D


def places(D):
    """For a block of 16 rows: byte and shift of each number of keys and of values [16, D], and the scales' bytes
    [16, D / 32] of both."""
    nb = D // 32
    kb, ks, vb, vs = (torch.zeros((16, D), dtype=torch.long) for _ in range(4))
    kc, vc = (torch.zeros((16, nb), dtype=torch.long) for _ in range(2))
    for r in range(16):
        for d in range(D):
            b, t, j, h = d // 32, d % 32 // 8, d % 8 // 2, d % 2
            bit = 32 * ((4 * r + t) * nb + b) + 16 * h + 4 * j
            kb[r, d], ks[r, d] = bit // 8, bit % 8
            u, g, i, p, t, c = d // 32, d % 32 // 4, d % 4, r // 8, r % 8 // 2, r % 2
            bit = 32 * (((8 * p + g) * 4 + t) * nb + u) + 16 * c + 4 * i
            vb[r, d], vs[r, d] = 8 * D + bit // 8, bit % 8
        for b in range(nb):
            kc[r, b], vc[r, b] = 16 * D + r * nb + b, 16 * D + 16 * nb + (r // 2) * 2 * nb + 2 * b + r % 2
    return kb, ks, vb, vs, kc, vc


def round4(x):
    """Numbers -7 .. 7 and scale bytes of rows [..., D], from their values in 64 bits."""
    y = x.double().unflatten(-1, (-1, 32))
    grid = torch.tensor(SCALES[:MOST + 1], dtype=torch.float64, device=x.device)
    code = (7 * grid < y.abs().amax(-1)[..., None]).sum(-1).clamp(max=MOST)
    d = grid[code][..., None]
    n = torch.where(d > 0, torch.round(y / torch.where(d > 0, d, 1.0)), 0.0).clamp(-7, 7)
    return n.flatten(-2), code


def value4(n, code):
    """The 64-bit values n d."""
    d = torch.tensor(SCALES, dtype=torch.float64, device=n.device)[code]
    return (n.double().unflatten(-1, (-1, 32)) * d[..., None]).flatten(-2)


def pack(k, v):
    """(n, code) of keys and of values, [P, R, H, D], as pages uint8 [P, bytes]."""
    (kn, kc), (vn, vc) = k, v
    P, R, H, D = kn.shape
    kb, ks, vb, vs, kp, vp = (t.to(kn.device) for t in places(D))
    blocks = torch.zeros((P, H, R // 16, block_bytes(D)), dtype=torch.long, device=kn.device)

    def rows(t):
        return t.permute(0, 2, 1, 3).unflatten(2, (R // 16, 16)).flatten(3).long()

    for n, at, shift in ((kn + 8, kb, ks), (vn + 8, vb, vs)):
        blocks.scatter_add_(-1, at.flatten().expand(P, H, R // 16, -1), rows(n) << shift.flatten())
    for c, at in ((kc, kp), (vc, vp)):
        blocks.scatter_add_(-1, at.flatten().expand(P, H, R // 16, -1), rows(c))
    return blocks.to(torch.uint8).flatten(1)


def unpack(pages, R, H, D):
    """Pages uint8 [P, bytes] as 64-bit keys and values [P, R, H, D]."""
    kb, ks, vb, vs, kc, vc = (t.to(pages.device) for t in places(D))
    x = pages[:, :R // 16 * H * block_bytes(D)].reshape(-1, H, R // 16, block_bytes(D)).long()
    grid = torch.tensor(SCALES, dtype=torch.float64, device=pages.device)
    out = []
    for at, shift, code in ((kb, ks, kc), (vb, vs, vc)):
        n = ((x[..., at] >> shift) & 15).double() - 8
        y = n * grid[x[..., code]].repeat_interleave(32, -1)
        out.append(y.flatten(2, 3).transpose(1, 2))
    return out


def gather(pages, table, R, H, D, lens):
    """64-bit keys and values [n, width R, H, D] of the sequences, zeros on entries that are no page (only pages of rows
    below the lengths are looked at)."""
    n, width = table.shape
    k = torch.zeros((n, width * R, H, D), dtype=torch.float64, device=pages.device)
    v = torch.zeros_like(k)
    for i in range(n):
        for j in range(-(-max(0, min(int(lens[i]), width * R)) // R)):
            p = int(table[i, j])
            if 0 <= p < len(pages):
                kk, vv = unpack(pages[p:p + 1], R, H, D)
                k[i, j * R:(j + 1) * R], v[i, j * R:(j + 1) * R] = kk[0], vv[0]
    return k, v


def random_cache(n, width, R, H, D, seed, spare=3, std=1.0, device="cuda"):
    """A KV4 with its pages in no order, rows of normal numbers, and pages that no table names full of 0xFF."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    P = n * width + spare
    pages = torch.full((P, mq.mq_kv4_page_bytes(R, H, D)), 255, dtype=torch.uint8, device=device)
    order = torch.randperm(P, generator=g, device=device)[:n * width]
    k, v = (round4(torch.randn((n * width, R, H, D), generator=g, device=device) * std) for _ in range(2))
    if n * width:
        pages[order] = pack(k, v)
    return mq.KV4(pages, order.to(torch.int32).view(n, width), R, H, D)


def next_pages(table, length, frm, keep, add, n_pages, R, m):
    """mq_pages_next on lists: (table_out, len_out, status, copies)."""
    n, width = len(table), len(table[0]) if table else 0
    frm = list(range(m)) if frm is None else frm
    L, extra, rows, longs = [], [], [], 0
    for b in range(m):
        f = frm[b]
        have = min(max(length[f], 0), width * R) if 0 <= f < n else 0
        if keep is not None:
            have = min(have, max(keep[b], 0))
        more = 0 if add is None else max(add[b], 0)
        if have + more > width * R:
            more, longs = 0, longs + 1
        L.append(have)
        extra.append(more)
        used = -(-have // R)
        rows.append([table[f][j] if j < used else -1 for j in range(width)])
    holders = {}
    for b in range(m):
        for j in range(-(-L[b] // R)):
            if 0 <= rows[b][j] < n_pages:
                holders.setdefault(rows[b][j], []).append((b, j))
    inside = {b: L[b] // R for b in range(m) if extra[b] > 0 and L[b] % R}
    copy = set()
    for b, j in inside.items():
        p = rows[b][j]
        if not 0 <= p < n_pages or len(holders[p]) == 1:
            continue
        writers = [x for x, y in holders[p] if x in inside and inside[x] == y]
        if len(writers) == len(holders[p]) and min(writers) == b:
            continue
        copy.add(b)
    free = [p for p in range(n_pages) if p not in holders]
    want = sum(-(-(L[b] + extra[b]) // R) - -(-L[b] // R) for b in range(m)) + len(copy)
    if want > len(free):
        return rows, L, [want - len(free), len(free), longs], []
    left = list(free)
    copies = []
    for b in range(m):
        if b in copy:
            p = left.pop(0)
            copies.append((rows[b][inside[b]], p))
            rows[b][inside[b]] = p
        for j in range(-(-L[b] // R), -(-(L[b] + extra[b]) // R)):
            rows[b][j] = left.pop(0)
    return rows, [x + y for x, y in zip(L, extra)], [0, len(left), longs], copies


def compact_pages(table, length, n_pages, R):
    """mq_pages_compact on lists: (table_out, where, live, moves)."""
    width = len(table[0]) if table else 0
    used = [-(-min(max(x, 0), width * R) // R) for x in length]
    live = sorted({p for row, u in zip(table, used) for p in row[:u] if 0 <= p < n_pages})
    U = len(live)
    where = [-1] * n_pages
    for p in live:
        where[p] = p
    moves = list(zip([p for p in live if p >= U], [p for p in range(U) if where[p] < 0]))
    for a, b in moves:
        where[a] = b
    out = [[(where[p] if 0 <= p < n_pages else p) if j < u else -1 for j, p in enumerate(row)] for row, u in zip(table, used)]
    return out, where, U, moves
