"""Plain 64-bit references of the serving operators (rotary positions, the KV
cache's rows, attention of drafted trees, residual norms), on whatever device
the inputs are on."""
import math

import torch

F16, Q8 = 16, 1


def inv_freqs(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def rotate(x, pos, inv, interleaved, mscale=1.0):
    """x [heads, M, D] in 64 bits, rotated; and the sum of magnitudes |a| + |b|
    of each value's pair (0 where nothing turns)."""
    x = x.double().clone()
    size = torch.zeros_like(x)
    rot = 2 * inv.numel()
    angle = pos.double()[:, None] * inv.to(x.device)
    c, s = angle.cos() * mscale, angle.sin() * mscale
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mscale)
    return x, size


def round_up_half(x):
    """64-bit x >= 0 rounded up to fp16."""
    h = x.to(torch.float16)
    low = h.double() < x
    return torch.where(low, (h.view(torch.int16) + 1).view(torch.float16), h)


def encode(x):
    """Q8_0 (d fp16 [..., nb], q int8 [..., nb, 32]) of 64-bit rows [..., D]."""
    y = x.double().unflatten(-1, (-1, 32))
    d = round_up_half(y.abs().amax(-1) / 127)
    dd = d.double()[..., None]
    q = torch.where(dd > 0, torch.round(y / torch.where(dd > 0, dd, 1.0)), 0.0)
    return d, q.to(torch.int8)


def pack(d, q):
    b = torch.cat([d[..., None].contiguous().view(torch.uint8), q.view(torch.uint8)], -1)
    return b.flatten(-2)


def values(rows, codec):
    """Cache rows -> their values in 64 bits (Q8_0: each rounded to fp16)."""
    if codec == F16:
        return rows.double()
    b = rows.unflatten(-1, (-1, 34))
    d = b[..., :2].contiguous().view(torch.float16).double()
    q = b[..., 2:].contiguous().view(torch.int8).double()
    return (q * d).to(torch.float16).double().flatten(-2)


def used_and_seen(parents):
    """Per sequence: used[i], and for each node the list of nodes it sees."""
    used, seen = [], []
    for i, a in enumerate(parents):
        if a == -1:
            used.append(True)
            seen.append([i])
        elif 0 <= a < i and used[a]:
            used.append(True)
            seen.append(seen[a] + [i])
        else:
            used.append(False)
            seen.append([])
    return used, seen


def tree_attention(q, kc, vc, codec, past, parents, scale):
    """(o, tol): O [B N, H D] in 64 bits, from a loop over sequences, and the
    tolerance of each value (see the test module)."""
    h, rows, d = q.shape
    b, hkv, c, _ = kc.shape
    n = rows // b
    o = torch.zeros(b, n, h, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    g = h // hkv
    for s in range(b):
        p = min(max(int(past[s]), 0), c)
        used, seen = used_and_seen([int(v) for v in parents[s]])
        for i in range(n):
            if not used[i]:
                continue
            keys = list(range(p)) + [p + a for a in seen[i] if p + a < c]
            if not keys:
                continue
            idx = slice(0, p) if len(keys) == p else torch.tensor(keys, device=q.device)
            k = values(kc[s][:, idx], codec).repeat_interleave(g, 0)
            v = values(vc[s][:, idx], codec).repeat_interleave(g, 0)
            x = torch.einsum("hd,hjd->hj", q[:, s * n + i].double(), k) * scale
            w = torch.softmax(x, -1)
            o[s, i] = torch.einsum("hj,hjd->hd", w, v)
            mag = torch.einsum("hj,hjd->hd", w, v.abs())
            big = v.abs().amax(1)
            span = (torch.einsum("hd,hjd->hj", q[:, s * n + i].double().abs(), k.abs()) * abs(scale)).amax(-1)
            tol[s, i] = (2.0 ** -11 + 2.0 ** -20 + 2 * span[:, None] * 2.0 ** -22) * mag \
                + 2.0 ** -11 * o[s, i].abs() + 2.0 ** -25 * (len(keys) * big + 1)
    return o.reshape(rows, h * d), tol.reshape(rows, h * d)


def norm_residual(h, r, w_pre, w_post, gate, res_scale, branch_scale, eps):
    r = r.double()
    if h is not None:
        u = h.double()
        if w_post is not None:
            u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * w_post.double()
        if gate is not None:
            u = u * gate.double()
        r = res_scale * r + branch_scale * u
    y = None
    if w_pre is not None:
        y = r / (r.square().mean(-1, keepdim=True) + eps).sqrt() * w_pre.double()
    return y, r
