"""Cases of the operators of a serving loop over a paged KV cache: rotary
positions of several axes (images, video) with the cache written, block tables
and slots planned from request lengths, attention of one new token a sequence
over the pages, and drafted trees of tokens verified against the target's
probabilities.

Every case has its plain form (elementary torch operations in 32 bits; in 64
where a decision stands beside a border) and the framework's call; ``own``
chooses which one ``run`` makes.  ``exact`` computes the same outputs in 64
bits.
"""
import math

import torch

own = False

F16, Q8 = "f16", "q8_0"
HALF, INTERLEAVED = "half", "interleaved"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A decode step of 16 sequences that hold images: 32 heads of queries
        # turned by time, height and width (latency).
        _turn("turn_step", 32, 16, 128, 128, HALF, "16,24,24", False, True),
        # A prompt of 8192 video tokens, the pairs dealt out over the axes in
        # turn.
        _turn("turn_video", 32, 8192, 128, 128, HALF, "24,20,20", True, True),
        # A prompt of 4000 image tokens: queries turned, keys turned and
        # written with the values to Q8_0 pages, and the rows read back.
        _image("write_image_q8_0", Q8, 8, 4, 128, 128, HALF, "16,24,24", False, 64, 4000),
        # A decode step's plan: 64 sequences of one new token each.
        _plan("plan_step", 64, 16, 500, 1, 64, 0),
        # A step with prompts: 256 sequences of up to 127 new tokens, 1 in 16
        # has ended, room for 16384 tokens.
        _plan("plan_prompts", 256, 64, 4000, 127, 16384, 16),
        # The first new token after a short prompt, one sequence.
        _paged("token_first_f16", F16, 32, 8, 128, 1, 16, 300, 300, False),
        # 32 sequences over 500 to 8100 keys, Q8_0 pages.
        _paged("token_batch_q8_0", Q8, 32, 8, 128, 32, 64, 500, 8100, False),
        # 64 sequences in a batch padded with empty ones, heads of 64 in
        # groups of eight, small pages.
        _paged("token_batch_f16", F16, 32, 4, 64, 64, 16, 100, 4000, True),
        # One very long document.
        _paged("token_long_f16", F16, 32, 8, 128, 1, 256, 131001, 131001, False),
        # One sequence, a chain of four drafted tokens behind the last one.
        _verify("verify_chain", 1, 5, 32000, "f32", True),
        # 16 sequences with trees of 7 drafted tokens.
        _verify("verify_trees", 16, 8, 128000, "f32", False),
        # A large batch of short chains, fp16 probabilities, rows of an odd
        # length.
        _verify("verify_batch", 96, 4, 50001, "f16", True),
    ]


def _named(name, **case):
    return dict(case, name=name) if name else case


def _turn(name, heads, rows, dim, rot, layout, sections, dealt, by_token):
    return _named(name, op="turn", heads=heads, rows=rows, dim=dim, rot=rot, layout=layout, sections=sections,
                  dealt=dealt, by_token=by_token)


def _image(name, codec, kv_heads, group, dim, rot, layout, sections, dealt, page, rows):
    return _named(name, op="image", codec=codec, kv_heads=kv_heads, group=group, dim=dim, rot=rot, layout=layout,
                  sections=sections, dealt=dealt, page=page, rows=rows)


def _plan(name, batch, page, most, each, tokens, ended):
    return _named(name, op="plan", batch=batch, page=page, most=most, each=each, tokens=tokens, ended=ended)


def _paged(name, codec, heads, kv_heads, dim, batch, page, least, most, padded):
    return _named(name, op="paged", codec=codec, heads=heads, kv_heads=kv_heads, dim=dim, batch=batch, page=page,
                  least=least, most=most, padded=padded)


def _verify(name, batch, nodes, words, dtype, chain):
    return _named(name, op="verify", batch=batch, nodes=nodes, words=words, dtype=dtype, chain=chain)


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def _split(rng, pairs):
    """Pairs of a row dealt to two or three axes, the first with the most."""
    n = rng.choice([2, 3, 3])
    rest = [rng.randint(1, pairs // (n + 1)) for _ in range(n - 1)]
    return ",".join(str(v) for v in [pairs - sum(rest)] + rest)


def draw(rng):
    op = rng.choice(["turn", "image", "plan", "paged", "paged", "paged", "verify", "verify"])
    dim = rng.choice([64, 128])
    rot = 16 * rng.randint(1, dim // 16)
    layout = rng.choice([HALF, INTERLEAVED])
    codec = rng.choice([F16, Q8])
    page = 8 * rng.choice([1, 2, 3, 4, 8, 16, 32])
    dealt = rng.random() < 0.5
    if op == "turn":
        heads = _log(rng, 1, 64)
        rows = _log(rng, 1, 8192 * 32 * 128 // (heads * dim) if heads * dim > 4096 else 8192)
        return _turn(None, heads, rows, dim, rot, layout, _split(rng, rot // 2), dealt, rng.random() < 0.5)
    if op == "image":
        return _image(None, codec, _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 8]), dim, rot, layout,
                      _split(rng, rot // 2), dealt, page, _log(rng, 1, 4000))
    if op == "plan":
        batch = _log(rng, 1, 512)
        each = _log(rng, 1, max(1, 16384 // batch))
        return _plan(None, batch, page, _log(rng, 1, 4000), each, _log(rng, max(1, batch * each // 2), batch * each + 16),
                     rng.choice([0, 3, 16]))
    if op == "paged":
        kv_heads, group = _log(rng, 1, 8), rng.choice([1, 2, 3, 4, 4, 6, 8, 12, 16])
        batch = _log(rng, 1, 128)
        most = _log(rng, 1, min(32000, 128000 // batch))
        return _paged(None, codec, kv_heads * group, kv_heads, dim, batch, page, _log(rng, 1, most), most,
                      rng.random() < 0.5)
    batch, nodes = _log(rng, 1, 64), _log(rng, 1, 24)
    words = _log(rng, 16, min(200000, 16000000 // (batch * nodes)))
    return _verify(None, batch, nodes, words, rng.choice(["f32", "f32", "f16"]), rng.random() < 0.5)


# Keys of sequence b, spread over [least, most]; a padded batch holds an empty
# sequence in eight.

def _lengths(case):
    n, lo, hi = case["batch"], case["least"], case["most"]
    out = [hi if n == 1 else lo + (hi - lo) * ((5 * b + 2) % n) // max(1, n - 1) for b in range(n)]
    return [0 if case["padded"] and b % 8 == 7 else v for b, v in enumerate(out)]


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _normal(g, shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _pool(g, case, pages):
    """One page pool [pages, kv_heads, page, row], every row filled."""
    x = _normal(g, (pages, case["kv_heads"], case["page"], case["dim"]))
    return x if case["codec"] == F16 else _pack(x.float())


def _ints(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


def _frequencies(rot):
    """Radians per position in 64 bits, and the framework's table of the same:
    turns per position in units of 2^-64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    inv = 10000.0 ** (-2.0 * i / rot)
    return inv, torch.round(inv / (2 * math.pi) * 2.0 ** 64).to(torch.int64)


def _axes(case):
    """The axis of each pair: sections one after the other, or dealt out in
    turn (what the later axes leave is the first one's)."""
    n = [int(v) for v in case["sections"].split(",")]
    if not case["dealt"]:
        return [a for a, c in enumerate(n) for _ in range(c)]
    return [i % len(n) if i < len(n) * n[i % len(n)] else 0 for i in range(sum(n))]


def _places(g, rows):
    """Positions [time, height, width] of some text and a grid of patches."""
    base = 1000 + torch.randint(0, 5000, (1,), generator=g, device="cuda")
    text = rows // 8
    side = max(1, int((rows - text) ** 0.4))
    i = torch.arange(rows, device="cuda")
    k = (i - text).clamp(min=0)
    grid = torch.stack([k // (side * side), k // side % side, k % side]) + text
    return (base + torch.where(i < text, i, grid)).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op in ("turn", "image"):
        axes, m = _axes(case), case["rows"]
        s["inv"], s["freqs"] = _frequencies(case["rot"])
        s["axes"] = _ints(axes)
        s["pos"] = _places(g, m)[:max(axes) + 1].contiguous()
    if op == "turn":
        h, d = case["heads"], case["dim"]
        # by_token: the rows of a row-major projection, seen head by head
        s["x"] = _normal(g, (m, h, d)).transpose(0, 1) if case["by_token"] else _normal(g, (h, m, d))
    elif op == "image":
        hk, d, page = case["kv_heads"], case["dim"], case["page"]
        qkv = _normal(g, ((case["group"] + 2) * hk, m, d))   # the fused projection's head-major rows
        nq = case["group"] * hk
        s["q"], s["k"], s["v"] = qkv[:nq], qkv[nq:nq + hk], qkv[nq + hk:]
        pages = 2 * ((m + page - 1) // page) + 1
        row = torch.arange(m, device="cuda")
        s["slots"] = (torch.randperm(pages, generator=g, device="cuda")[row // page] * page + row % page).to(torch.int32)
        s["kc"], s["vc"] = _pool(g, case, pages), _pool(g, case, pages)
    elif op == "plan":
        b, page = case["batch"], case["page"]
        past = torch.randint(0, case["most"] + 1, (b,), generator=g, device="cuda")
        new = torch.randint(1, case["each"] + 1, (b,), generator=g, device="cuda")
        held = (past + page - 1) // page
        width = (case["most"] + case["each"] + page - 1) // page
        pages = b * width + 3
        ids = torch.randperm(pages, generator=g, device="cuda")
        used = torch.arange(width, device="cuda") < held[:, None]
        taken = int(held.sum())
        s["table"] = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        s["table"][used] = ids[:taken].to(torch.int32)
        s["free"] = torch.cat([ids[taken:], ids[:taken]]).to(torch.int32)   # behind the free ones: stale ids
        s["n_free"] = _ints([pages - taken])
        if case["ended"]:
            new[torch.arange(b, device="cuda") % case["ended"] == 1] = -1
        s["past"], s["new"], s["held"] = past.to(torch.int32), new.to(torch.int32), held.to(torch.int32)
    elif op == "paged":
        b, page = case["batch"], case["page"]
        s["q"] = _normal(g, (case["heads"], b, case["dim"]))
        lengths = torch.tensor(_lengths(case), device="cuda")
        width = (case["most"] + page - 1) // page + 2
        held = (lengths + page - 1) // page
        need = sum((n + page - 1) // page for n in _lengths(case))
        pages = need + need // 8 + 8
        used = torch.arange(width, device="cuda") < held[:, None]
        s["table"] = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        s["table"][used] = torch.randperm(pages, generator=g, device="cuda")[:need].to(torch.int32)
        s["lengths"] = lengths.to(torch.int32)
        s["kc"], s["vc"] = _pool(g, case, pages), _pool(g, case, pages)
    else:
        b, n, v = case["batch"], case["nodes"], case["words"]
        # a draft model's scores are the target's with an error
        score = torch.randn((b, n, v), generator=g, device="cuda") * 2.5
        s["target"] = _softmax(score)
        s["draft"] = _softmax(score + 0.8 * torch.randn((b, n, v), generator=g, device="cuda"))
        i = torch.arange(n, device="cuda")
        back = torch.randint(1, 4, (b, n), generator=g, device="cuda")
        parents = (i - 1).expand(b, n) if case["chain"] else torch.where(i > 0, (i - back).clamp(min=0), -1)
        # each drafted token comes from its parent's distribution
        rows = torch.gather(s["draft"].cumsum(-1), 1, parents.clamp(min=0)[:, :, None].expand(b, n, v))
        at = torch.rand((b, n, 1), generator=g, device="cuda") * rows[:, :, -1:]
        s["tokens"] = torch.searchsorted(rows.contiguous(), at, right=True).clamp(max=v - 1)[:, :, 0].to(torch.int32)
        s["parents"] = parents.to(torch.int32).contiguous()
        s["u"] = torch.rand((b, n), generator=g, device="cuda")
        if case["dtype"] == "f16":
            s["target"], s["draft"] = s["target"].half(), s["draft"].half()
    return s


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


# ---------------------------------------------------------------- plain forms

def _pack(x):
    """Rows [..., D] in 32 bits -> Q8_0 blocks [..., D / 32 * 34]: the scale
    is amax / 127 rounded up to fp16, the codes are x / scale to nearest."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    want = blocks.abs().amax(-1, keepdim=True) / 127.0
    d = want.half()
    d = torch.where(d.float() < want, (d.view(torch.int16) + 1).view(torch.float16), d)
    q = torch.where(d > 0, torch.round(blocks / d.float()), 0.0).to(torch.int8)
    return torch.cat([d.view(torch.uint8), q.view(torch.uint8)], -1).reshape(*x.shape[:-1], -1)


def _unpack(rows):
    """Q8_0 blocks -> their fp16 values in 32 bits (fp16 rows: as they are)."""
    if rows.dtype == torch.float16:
        return rows.float()
    blocks = rows.reshape(*rows.shape[:-1], rows.shape[-1] // 34, 34)
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    q = blocks[..., 2:].contiguous().view(torch.int8).float()
    return (q * d).half().float().reshape(*rows.shape[:-1], -1)


def _rotate(x, s):
    """x [heads, rows, D] in 32 bits, pair i of its first rot values turned by
    the position of its axis."""
    rot, angle = s["rot"], s["pos"][s["axes"].long()].double().transpose(0, 1) * s["inv"]
    cos, sin = angle.cos().float(), angle.sin().float()
    t, rest = x[..., :rot], x[..., rot:]
    if s["layout"] == HALF:
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([t, rest], -1)


def _plain_image(s):
    page, slot = s["page"], s["slots"].long()
    k, v = _rotate(s["k"].float(), s), s["v"].float()
    out = {"q": _rotate(s["q"].float(), s).half()}
    for name, pool, rows in (("k", s["kc"], k), ("v", s["vc"], v)):
        rows = rows.half() if s["codec"] == F16 else _pack(rows)
        pool[slot // page, :, slot % page] = rows.transpose(0, 1)
        out[name] = _unpack(pool[slot // page, :, slot % page].transpose(0, 1)).half()
    return out


def _plain_plan(s):
    page, t, (b, width), pages = s["page"], s["tokens"], s["table"].shape, s["free"].numel()
    past, new, held, table = s["past"].long(), s["new"].long(), s["held"].long(), s["table"].long()
    n_free = s["n_free"].long()
    ends = new.clamp(min=0).cumsum(0).clamp(max=t)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    n = starts[1:] - starts[:-1]
    live = (new >= 0)[:, None]
    want = ((past + n + page - 1) // page).clamp(max=width)
    take = torch.where(new >= 0, (want - held).clamp(min=0), 0)
    first = take.cumsum(0) - take
    got = (n_free - first).clamp(min=0).minimum(take)
    j = torch.arange(width, device="cuda")
    k = first[:, None] + j - held[:, None]                 # which page of this call entry j is
    page_of = torch.where(k < n_free, s["free"].long()[(n_free - 1 - k).clamp(0, pages - 1)], -1)
    fresh = live & (j >= held[:, None]) & (j < (held + take)[:, None])
    back = ~live & (j < held[:, None])                     # the pages of sequences that have ended
    done = torch.where(fresh, page_of, torch.where(back, -1, table))
    # they go on top of what is left, in their order
    left = n_free - got.sum()
    order = (back.flatten().cumsum(0) - 1).view(b, width)
    to = torch.where(back, left + order, pages)
    free = torch.cat([s["free"], s["free"][:1]])
    free[to.flatten()] = table.flatten().to(torch.int32)
    i = torch.arange(t, device="cuda")
    seq = torch.searchsorted(ends, i, right=True).clamp(max=b - 1)
    real = i < ends[-1]
    pos = torch.where(real, past[seq] + i - starts[seq], 0)
    at = pos // page
    entry = done[seq, at.clamp(max=width - 1)]
    slots = torch.where(real & (at < width) & (entry >= 0), entry * page + pos % page, -1)
    holds = torch.where(new >= 0, held + got, 0)
    lengths = torch.where(new >= 0, (past + n).minimum(holds * page), 0)
    s["table"].copy_(done)
    s["held"].copy_(holds)
    s["free"].copy_(free[:-1])
    s["n_free"].copy_(left + back.sum())
    return {"slots": slots.int(), "pos": pos.int(), "lengths": lengths.int(), "starts": starts.int(),
            "table": s["table"], "held": s["held"], "free": s["free"], "n_free": s["n_free"]}


def _plain_paged(s):
    h, b, d = s["q"].shape
    hk, page, width = s["kv_heads"], s["page"], s["table"].shape[1]
    at = s["table"].long().clamp(min=0)
    keys = torch.arange(width * page, device="cuda")
    seen = (keys < s["lengths"].long()[:, None])[:, None, None]             # [b, 1, 1, keys]
    q = s["q"].float().reshape(hk, h // hk, b, d).permute(2, 0, 1, 3)       # [b, hk, group, d]

    def rows(pool):
        return _unpack(pool[at].transpose(1, 2).reshape(b, hk, width * page, -1))
    score = torch.where(seen, q @ rows(s["kc"]).transpose(2, 3) * d ** -0.5, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = (p @ rows(s["vc"])) / torch.where(total > 0, total, 1.0)
    return o.reshape(b, h * d).half()


def _plain_verify(s):
    b, n, v = s["target"].shape
    row = torch.arange(b, device="cuda")
    parents, tokens, u = s["parents"].long(), s["tokens"].long(), s["u"].double()
    node, count = torch.zeros_like(row), torch.ones_like(row)
    off, mass = torch.zeros_like(u[:, 0]), torch.ones_like(u[:, 0])
    path = torch.full_like(parents, -1)
    path[:, 0] = 0
    for i in range(1, n):
        child = parents[:, i] == node
        p, q = (s[x][row, node, tokens[:, i]].double() for x in ("target", "draft"))
        yes = child & (u[:, i] * mass * q < p - off * q)
        no = child & ~yes
        path[row, count.clamp(max=n - 1)] = torch.where(yes, i, path[row, count.clamp(max=n - 1)])
        count = count + yes
        off = torch.where(no, off + mass, off)
        rest = (s["target"][row, node].double() - off[:, None] * s["draft"][row, node].double()).clamp(min=0)
        mass = torch.where(yes, 1.0, torch.where(no, rest.sum(-1), mass))
        off = torch.where(yes, 0.0, off)
        node = torch.where(yes, i, node)
    p = s["target"][row, node].double()
    rest = (p - off[:, None] * s["draft"][row, node].double()).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    upto = rest.cumsum(-1)
    token = (upto <= u[:, :1] * upto[:, -1:]).sum(-1).clamp(max=v - 1)
    return {"path": path.int(), "count": count.int(), "token": token.int()}


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s)
    if op == "turn":
        return _rotate(s["x"].float(), s).half()
    return {"image": _plain_image, "plan": _plain_plan, "paged": _plain_paged, "verify": _plain_verify}[op](s)


def _own(s):
    import swiglu_block_quantized_gb300 as m
    op = s["op"]
    if op == "plan":
        slots, pos, lengths, starts = m.page_plan(s["past"], s["new"], s["table"], s["held"], s["free"], s["n_free"],
                                                  s["page"], s["tokens"])
        return {"slots": slots, "pos": pos, "lengths": lengths, "starts": starts, "table": s["table"],
                "held": s["held"], "free": s["free"], "n_free": s["n_free"]}
    if op == "verify":
        path, count, token = m.verify_tree(s["target"], s["draft"], s["tokens"], s["parents"], s["u"])
        return {"path": path, "count": count, "token": token}
    layout = m.ROPE_HALF if s.get("layout") == HALF else m.ROPE_INTERLEAVED
    if op == "turn":
        return m.rope(s["x"], s["pos"], s["freqs"], layout=layout, axes=s["axes"])
    codec = m.KV_F16 if s["codec"] == F16 else m.Q8_0
    if op == "paged":
        return m.attention_paged(s["q"], s["kc"], s["vc"], codec, s["table"], s["lengths"])
    q = m.kv_write(s["k"], s["v"], s["kc"], s["vc"], codec, s["slots"], pos=s["pos"], freqs=s["freqs"], layout=layout,
                   axes=s["axes"], q=s["q"])
    k, v = m.kv_read(s["kc"], s["vc"], codec, s["slots"])
    return {"q": q, "k": k, "v": v}


# ---------------------------------------------------------------- bytes and operations

def _row(case):
    return 2 * case["dim"] if case["codec"] == F16 else case["dim"] // 32 * 34


def work(case):
    op = case["op"]
    if op == "turn":
        n = case["heads"] * case["rows"]
        return {"bytes": 4 * n * case["dim"] + 12 * case["rows"], "flops": 3 * n * case["rot"]}
    if op == "image":
        n = case["kv_heads"] * case["rows"]
        # K and V in, their rows out and read back, and the queries
        return {"bytes": 2 * n * (4 * case["dim"] + 2 * _row(case)) + 4 * case["group"] * n * case["dim"],
                "flops": n * (3 * case["rot"] * (1 + case["group"]) + 6 * case["dim"])}
    if op == "plan":
        # lengths and counts of every sequence, a table entry and two numbers
        # for every token
        b, t = case["batch"], case["tokens"]
        return {"bytes": 4 * (6 * b + 3 * t), "flops": b + t}
    if op == "paged":
        keys = sum(_lengths(case))
        return {"bytes": 2 * case["kv_heads"] * keys * _row(case) + 4 * case["heads"] * case["batch"] * case["dim"],
                "flops": 4 * case["heads"] * case["dim"] * keys}
    # a row of the target's probabilities, and of the draft's where there is one
    n = case["batch"] * case["words"] * (2 if case["nodes"] > 1 else 1)
    return {"bytes": n * (4 if case["dtype"] == "f32" else 2), "flops": 3 * n}


# ---------------------------------------------------------------- 64 bits

def _e_turn(x, s):
    theta = s["inv"][:, None] * s["pos"].to(torch.float64)[s["axes"].long()]
    z = torch.polar(torch.ones_like(theta), theta).T
    out, r = x.to(torch.float64).clone(), s["rot"]
    first = slice(0, r // 2) if s["layout"] == HALF else slice(0, r, 2)
    second = slice(r // 2, r) if s["layout"] == HALF else slice(1, r, 2)
    w = torch.complex(out[..., first].clone(), out[..., second].clone()) * z
    out[..., first], out[..., second] = w.real, w.imag
    return out


def _e_stored(x, codec):
    """What a cache row holds of x (64 bits), as values: x itself but for a
    last rounding (fp16), or code times scale (Q8_0)."""
    if codec == F16:
        return x
    y = x.unflatten(-1, (-1, 32))
    want = y.abs().max(-1, keepdim=True).values / 127
    d = want.to(torch.float16)
    d = torch.where(d.to(torch.float64) < want, (d.view(torch.int16) + 1).view(torch.float16), d).to(torch.float64)
    q = torch.where(d > 0, torch.round(y / d), torch.zeros_like(y))
    return (q * d).to(torch.float16).to(torch.float64).flatten(-2)


def _e_values(rows, codec):
    if codec == F16:
        return rows.to(torch.float64)
    b = rows.unflatten(-1, (-1, 34))
    d = (b[..., 0].to(torch.int32) + 256 * b[..., 1].to(torch.int32)).to(torch.int16).view(torch.float16)
    q = b[..., 2:].to(torch.int32)
    q = torch.where(q > 127, q - 256, q).to(torch.float64)
    return (q * d.to(torch.float64)[..., None]).to(torch.float16).to(torch.float64).flatten(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "turn":
        return _e_turn(s["x"], s)
    if op == "image":
        return {"q": _e_turn(s["q"], s), "k": _e_stored(_e_turn(s["k"], s), s["codec"]),
                "v": _e_stored(s["v"].to(torch.float64), s["codec"])}
    if op == "plan":
        return _e_plan(s)
    if op == "paged":
        return _e_paged(case, s)
    return _e_verify(s)


def _e_plan(s):
    page, room, pages = s["page"], s["tokens"], s["free"].numel()
    table, held, free = (s[x].cpu().tolist() for x in ("table", "held", "free"))
    stack, width = int(s["n_free"]), len(table[0])
    slots, pos, lengths, starts, ended = [], [], [], [0], []
    for b, (past, new) in enumerate(zip(s["past"].tolist(), s["new"].tolist())):
        if new < 0:
            ended += table[b][:held[b]]
            table[b][:held[b]] = [-1] * held[b]
            held[b] = 0
            lengths.append(0)
            starts.append(starts[-1])
            continue
        new = min(new, room - starts[-1])
        starts.append(starts[-1] + new)
        for j in range(held[b], min(width, -(-(past + new) // page))):
            table[b][j] = -1
            if stack:
                stack -= 1
                table[b][j] = free[stack]
                held[b] += 1
        for p in range(past, past + new):
            fits = p // page < width and table[b][p // page] >= 0
            slots.append(table[b][p // page] * page + p % page if fits else -1)
            pos.append(p)
        lengths.append(min(past + new, held[b] * page))
    free[stack:stack + len(ended)] = ended
    rest = room - len(slots)
    out = {"slots": slots + [-1] * rest, "pos": pos + [0] * rest, "lengths": lengths, "starts": starts, "table": table,
           "held": held, "free": free[:pages], "n_free": [stack + len(ended)]}
    return {k: _ints(v) for k, v in out.items()}


def _e_paged(case, s):
    h, b, d = s["q"].shape
    page, group = case["page"], h // case["kv_heads"]
    out = torch.zeros(b, h, d, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        at = s["table"][i].long()[j // page]
        k, v = (_e_values(x[at, :, j % page], case["codec"]).repeat_interleave(group, 1) for x in (s["kc"], s["vc"]))
        a = torch.softmax(torch.einsum("hd,jhd->hj", s["q"][:, i].to(torch.float64), k) / math.sqrt(d), -1)
        out[i] = torch.einsum("hj,jhd->hd", a, v)
    return out.reshape(b, h * d)


def _e_verify(s):
    b, n, v = s["target"].shape
    parents, tokens, u = (s[x].cpu().tolist() for x in ("parents", "tokens", "u"))
    path, count, token = [], [], []
    for i in range(b):
        node, kept, left = 0, [0], None
        for c in range(1, n):
            if parents[i][c] != node:
                continue
            q = s["draft"][i, node].to(torch.float64)
            if left is None:
                left, share = s["target"][i, node].to(torch.float64), 1.0
            x = tokens[i][c]
            if u[i][c] * share * float(q[x]) < float(left[x]):
                node, left = c, None
                kept.append(c)
            else:
                left = torch.relu(left - share * q)        # what the target has above the draft
                share = float(left.sum())
        if left is None:
            left = s["target"][i, node].to(torch.float64)
        if not float(left.sum()) > 0:
            left = s["target"][i, node].to(torch.float64)
        sums = torch.cumsum(left, 0)
        token.append(int(torch.searchsorted(sums, u[i][0] * sums[-1:], right=True).clamp(max=v - 1)))
        path.append(kept + [-1] * (n - len(kept)))
        count.append(len(kept))
    return {"path": _ints(path), "count": _ints(count), "token": _ints(token)}
