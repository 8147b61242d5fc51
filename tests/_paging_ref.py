"""Plain references of the paged serving loop's operators: page plans on the host,
attention over pages and verification of drafted trees in 64 bits."""
import torch

import _serving_ref as ref

I32 = 2 ** 31 - 1


def plan(past, new, table, held, free, n_free, page, tokens):
    """page_plan on lists; returns (slots, pos, lengths, starts, table, held, free, n_free)."""
    table, held, free = [list(r) for r in table], list(held), list(free)
    pages, width = len(free), len(table[0])
    n_free = min(max(n_free, 0), pages)
    slots, pos, lengths, starts, back, want_of = [], [], [], [0], [], []
    stack = n_free
    for b, n in enumerate(new):
        h = min(max(held[b], 0), width)
        p = max(past[b], 0)
        if n < 0:
            back += table[b][:h]
            table[b][:h] = [-1] * h
            held[b], n = 0, 0
            lengths.append(0)
        else:
            n = min(n, tokens - starts[-1])
            got = 0
            for j in range(h, min(width, -(-(p + n) // page))):
                if stack > 0:
                    stack -= 1
                    table[b][j] = free[stack]
                    got += 1
                else:
                    table[b][j] = -1
            held[b] = h + got
            lengths.append(min(p + n, held[b] * page))
            for q in range(p, p + n):
                e = table[b][q // page] if q // page < width else -1
                slots.append(e * page + q % page if 0 <= e < pages else -1)
                pos.append(min(q, I32))
        starts.append(starts[-1] + n)
    for i, x in enumerate(back):
        if stack + i < pages:
            free[stack + i] = x
    rest = tokens - len(slots)
    return (slots + [-1] * rest, pos + [0] * rest, lengths, starts, table, held, free, min(stack + len(back), pages))


def gather(pool, entries, n, codec):
    """Rows 0 .. n - 1 of a sequence as values [Hkv, n, D] in 64 bits, and which of them
    a page holds."""
    pages, _, page, _ = pool.shape
    j = torch.arange(n, device=pool.device)
    e = entries.long()[j // page]
    there = (e >= 0) & (e < pages)
    return ref.values(pool[e.clamp(0, pages - 1), :, j % page], codec).transpose(0, 1), there


def paged_attention(q, kc, vc, codec, table, lengths, scale):
    """(o, tol): O [B, H D] in 64 bits, and the tolerance of each value (that of
    _serving_ref.tree_attention)."""
    h, b, d = q.shape
    page, g = kc.shape[2], h // kc.shape[1]
    o = torch.zeros(b, h, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for s in range(b):
        n = min(max(int(lengths[s]), 0), table.shape[1] * page)
        if n == 0:
            continue
        k, there = gather(kc, table[s], n, codec)
        v, _ = gather(vc, table[s], n, codec)
        if not there.any():
            continue
        k, v = (x[:, there].repeat_interleave(g, 0) for x in (k, v))
        qs = q[:, s].double()
        w = torch.softmax(torch.einsum("hd,hjd->hj", qs, k) * scale, -1)
        o[s] = torch.einsum("hj,hjd->hd", w, v)
        mag = torch.einsum("hj,hjd->hd", w, v.abs())
        big = v.abs().amax(1)
        span = (torch.einsum("hd,hjd->hj", qs.abs(), k.abs()) * abs(scale)).amax(-1)
        tol[s] = (2.0 ** -11 + 2.0 ** -20 + 2 * span[:, None] * 2.0 ** -22) * mag \
            + 2.0 ** -11 * o[s].abs() + 2.0 ** -25 * (int(there.sum()) * big + 1)
    return o.reshape(b, h * d), tol.reshape(b, h * d)


def clean(x):
    x = x.double()
    return torch.where((x > 0) & (x < float("inf")), x, 0.0)


def verify(target, draft, tokens, parents, u):
    """(path, count, token) as lists, and how near the nearest decision was to its
    border, relative to what it compares."""
    b, n, v = target.shape
    tokens, parents, u = (x.cpu().tolist() for x in (tokens, parents, u))
    path, count, token, near = [], [], [], 1.0
    for s in range(b):
        if parents[s][0] != -1:
            path.append([-1] * n), count.append(0), token.append(-1)
            continue
        c, kept = 0, [0]
        rest, m, off = clean(target[s, 0]), 1.0, 0.0
        for i in range(1, n):
            x = tokens[s][i]
            if parents[s][i] != c or not 0 <= x < v:
                continue
            p, q = clean(target[s, c]), clean(draft[s, c])
            a, r = u[s][i] * m * float(q[x]), float(p[x] - off * q[x])
            if max(a, r) > 0:
                near = min(near, abs(a - r) / max(a, abs(r)))
            if a < r:
                c, m, off = i, 1.0, 0.0
                kept.append(i)
                rest = clean(target[s, c])
            else:
                off += m
                rest = (p - off * q).clamp(min=0)
                m = float(rest.sum())
        if not float(rest.sum()) > 0:
            rest = clean(target[s, c])
        sums = rest.cumsum(0)
        total = float(sums[-1])
        if total > 0:
            aim = u[s][0] * total
            t = min(int((sums <= aim).sum()), int(rest.nonzero().max()))
            near = min(near, float((sums[rest > 0] - aim).abs().min()) / total if u[s][0] > 0 else 1.0)
        else:
            t = -1
        path.append(kept + [-1] * (n - len(kept))), count.append(len(kept)), token.append(t)
    return path, count, token, near
