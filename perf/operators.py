"""Cases of the operators between a layer's projections: rotary positions, the
KV cache written (fp16 or Q8_0) and read back, attention of drafted trees of
tokens (or single tokens) over a batch of caches, and the norms around a block
with its gate and residual scale.

Every case has its plain form (elementary torch operations in 32 bits, angles
in 64) and the framework's call; ``own`` chooses which one ``run`` makes.
``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

F16, Q8 = "f16", "q8_0"
HALF, INTERLEAVED = "half", "interleaved"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # 16 sequences of one decode step, 8 drafted tokens each: the queries
        # of 32 heads of 128 get their positions (latency).
        _rope("rope_step", 32, 128, 128, 128, HALF, 5000, True, 1.0),
        # A prompt of 8192 tokens that continues a long document: far
        # positions, scaled frequencies with a magnitude factor.
        _rope("rope_prompt", 32, 8192, 128, 128, HALF, 250000, False, 1.2),
        # One decode step of 16 sequences with 8 drafted tokens: queries
        # rotated, keys rotated and written to an fp16 cache, one slot in 8
        # unused; interleaved pairs over half of a 64-wide head.
        _write("write_step_f16", F16, 8, 4, 64, 32, INTERLEAVED, 16, 8, 4096, True),
        # A prompt of 8000 tokens written to a Q8_0 cache.
        _write("write_prompt_q8_0", Q8, 8, 4, 128, 128, HALF, 1, 8000, 8192, False),
        # A few rows of an fp16 cache read back (a short shared prefix).
        _read("read_rows_f16", F16, 8, 64, 4, 2048, 200),
        # 16000 rows of a Q8_0 cache read back for another consumer.
        _read("read_prefix_q8_0", Q8, 8, 128, 2, 16384, 16000),
        # The first drafted tree after a short prompt, one sequence.
        _tree("tree_first_f16", F16, 32, 8, 128, 1, 8, 512, 300, 300),
        # 32 sequences of one new token each over ragged Q8_0 caches.
        _tree("token_batch_q8_0", Q8, 32, 8, 128, 32, 1, 8192, 500, 8100),
        # 8 sequences with trees of up to 24 drafted tokens, fp16 caches.
        _tree("tree_batch_f16", F16, 32, 8, 64, 8, 24, 8192, 1000, 8100),
        # One long sequence, 64 drafted tokens, Q8_0 cache.
        _tree("tree_long_q8_0", Q8, 32, 8, 128, 1, 64, 32768, 32500, 32500),
        # A decode step's 64 rows of 2048 between two blocks: pre-norm and
        # residual only, fp16 residual stream.
        _norm("norm_step", 64, 2048, False, False, "none", 1.0, 1.0),
        # A prompt's 8192 rows of 4096, norms on both sides of the block, a
        # gate per channel, fp32 residual stream.
        _norm("norm_prompt", 8192, 4096, True, True, "channel", 1.0, 0.5),
    ]


def _named(name, **case):
    return dict(case, name=name) if name else case


def _rope(name, heads, rows, dim, rot, layout, first, by_token, mscale):
    return _named(name, op="rope", heads=heads, rows=rows, dim=dim, rot=rot, layout=layout, first=first,
                  by_token=by_token, mscale=mscale)


def _write(name, codec, kv_heads, group, dim, rot, layout, batch, each, capacity, queries):
    return _named(name, op="write", codec=codec, kv_heads=kv_heads, group=group, dim=dim, rot=rot, layout=layout,
                  batch=batch, each=each, capacity=capacity, queries=queries)


def _read(name, codec, kv_heads, dim, batch, capacity, rows):
    return _named(name, op="read", codec=codec, kv_heads=kv_heads, dim=dim, batch=batch, capacity=capacity, rows=rows)


def _tree(name, codec, heads, kv_heads, dim, batch, nodes, capacity, least, most):
    return _named(name, op="tree", codec=codec, heads=heads, kv_heads=kv_heads, dim=dim, batch=batch, nodes=nodes,
                  capacity=capacity, least=least, most=most)


def _norm(name, rows, dim, res32, post, gate, res_scale, branch_scale):
    return _named(name, op="norm", rows=rows, dim=dim, res32=res32, post=post, gate=gate, res_scale=res_scale,
                  branch_scale=branch_scale)


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree", "norm"])
    dim = rng.choice([64, 128])
    rot = 16 * rng.randint(1, dim // 16)
    layout = rng.choice([HALF, INTERLEAVED])
    codec = rng.choice([F16, Q8])
    if op == "rope":
        heads = _log(rng, 1, 64)
        rows = _log(rng, 1, 8192 * 32 * 128 // (heads * dim) if heads * dim > 4096 else 8192)
        return _rope(None, heads, rows, dim, rot, layout, _log(rng, 1, 500000), rng.random() < 0.5,
                     rng.choice([1.0, 1.1, 1.3]))
    if op == "write":
        kv_heads, group = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 8])
        batch, each = _log(rng, 1, 32), _log(rng, 1, 64)
        if rng.random() < 0.4:
            batch, each = 1, _log(rng, 64, 4000)
        return _write(None, codec, kv_heads, group, dim, rot, layout, batch, each, 4 * ((each + _log(rng, 8, 4000)) // 4),
                      rng.random() < 0.5)
    if op == "read":
        capacity = 4 * _log(rng, 4, 4096)
        batch = _log(rng, 1, 8)
        return _read(None, codec, _log(rng, 1, 8), dim, batch, capacity, _log(rng, 1, min(16000, batch * capacity)))
    if op == "tree":
        kv_heads, group = _log(rng, 1, 8), rng.choice([1, 2, 4, 4, 8])
        batch, nodes = _log(rng, 1, 16), _log(rng, 1, 64)
        most = _log(rng, 8, max(16, min(16000, 32000 // batch)))
        capacity = 4 * ((most + nodes + 3) // 4 + _log(rng, 1, 64))
        return _tree(None, codec, kv_heads * group, kv_heads, dim, batch, nodes, capacity, _log(rng, 1, most), most)
    dim = 8 * _log(rng, 8, 2048)
    rows = _log(rng, 1, min(8192, 8192 * 4096 // dim))
    return _norm(None, rows, dim, rng.random() < 0.5, rng.random() < 0.5, rng.choice(["none", "channel", "row"]),
                 rng.choice([1.0, 0.8]), rng.choice([1.0, 0.25]))


# Sequence b of a batch: its keys so far, spread over [least, most], and its
# drafted nodes (the first sequence has them all).

def _pasts(case):
    n, lo, hi = case["batch"], case["least"], case["most"]
    return [hi if n == 1 else lo + (hi - lo) * ((5 * b + 2) % n) // max(1, n - 1) for b in range(n)]


def _counts(case):
    n = case["nodes"]
    return [n if b == 0 else max(1, n - (3 * b) % n) for b in range(case["batch"])]


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _cache(g, case):
    """One cache tensor [batch, kv_heads, capacity, row], every row filled."""
    shape = (case["batch"], case["kv_heads"], case["capacity"], case["dim"])
    x = _normal(g, shape)
    return x if case["codec"] == F16 else _pack(x.float())


def _frequencies(rot):
    """Radians per position in 64 bits, and the framework's table of the same:
    turns per position in units of 2^-64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    inv = 10000.0 ** (-2.0 * i / rot)
    return inv, torch.round(inv / (2 * math.pi) * 2.0 ** 64).to(torch.int64)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "rope":
        h, m, d = case["heads"], case["rows"], case["dim"]
        # by_token: the rows of a row-major projection, seen head by head
        s["x"] = _normal(g, (m, h, d)).transpose(0, 1) if case["by_token"] else _normal(g, (h, m, d))
        s["pos"] = (case["first"] + torch.randint(0, 64, (1,), generator=g, device="cuda") +
                    torch.arange(m, device="cuda")).to(torch.int32)
        s["inv"], s["freqs"] = _frequencies(case["rot"])
    elif op == "write":
        hk, d, b, n, c = case["kv_heads"], case["dim"], case["batch"], case["each"], case["capacity"]
        m = b * n
        qkv = _normal(g, ((case["group"] + 2) * hk, m, d))   # the fused projection's head-major rows
        nq = case["group"] * hk
        s["q"], s["k"], s["v"] = qkv[:nq], qkv[nq:nq + hk], qkv[nq + hk:]
        start = torch.randint(0, max(1, c - n), (b, 1), generator=g, device="cuda")
        j = start + torch.arange(n, device="cuda")
        s["pos"] = j.reshape(-1).to(torch.int32)
        slots = (torch.arange(b, device="cuda")[:, None] * c + j).reshape(-1)
        unused = (torch.arange(m, device="cuda") % 8 == 5) & (b > 1)   # padding of the batch
        s["slots"] = torch.where(unused, -1, slots).to(torch.int32)
        s["kc"], s["vc"] = _cache(g, case), _cache(g, case)
        s["inv"], s["freqs"] = _frequencies(case["rot"])
    elif op == "read":
        s["kc"], s["vc"] = _cache(g, case), _cache(g, case)
        n = case["batch"] * case["capacity"]
        first = torch.randint(0, n - case["rows"] + 1, (1,), generator=g, device="cuda")
        s["slots"] = (first + torch.arange(case["rows"], device="cuda")).to(torch.int32)
    elif op == "tree":
        b, n = case["batch"], case["nodes"]
        s["q"] = _normal(g, (case["heads"], b * n, case["dim"]))
        s["kc"], s["vc"] = _cache(g, case), _cache(g, case)
        s["past"] = torch.tensor(_pasts(case), dtype=torch.int32, device="cuda")
        # node i continues one of the up to 6 nodes before it, or the context
        i = torch.arange(n, device="cuda")
        back = torch.randint(1, 7, (b, n), generator=g, device="cuda")
        parents = torch.clamp(i - back, min=-1)
        count = torch.tensor(_counts(case), device="cuda")
        s["parents"] = torch.where(i < count[:, None], parents, -2).to(torch.int32)
    else:
        m, d = case["rows"], case["dim"]
        s["h"] = _normal(g, (m, d), 0.7)
        s["r"] = _normal(g, (m, d), 2.0, torch.float32 if case["res32"] else torch.float16)
        s["w_pre"] = (1.0 + 0.2 * _normal(g, (d,), dtype=torch.float32)).half()
        s["w_post"] = (1.0 + 0.2 * _normal(g, (d,), dtype=torch.float32)).half() if case["post"] else None
        shape = {"none": None, "channel": (d,), "row": (m, d)}[case["gate"]]
        s["g"] = _normal(g, shape, 0.5) if shape else None
    return s


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
    """Q8_0 blocks -> their fp16 values in 32 bits (an fp16 cache: as it is)."""
    if rows.dtype == torch.float16:
        return rows.float()
    blocks = rows.reshape(*rows.shape[:-1], rows.shape[-1] // 34, 34)
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    q = blocks[..., 2:].contiguous().view(torch.int8).float()
    return (q * d).half().float().reshape(*rows.shape[:-1], -1)


def _rotate(x, pos, inv, rot, layout, mscale):
    """x [heads, rows, D] in 32 bits (or 64) with its first rot values rotated."""
    angle = pos.double()[:, None] * inv
    cos, sin = (angle.cos() * mscale).to(x.dtype), (angle.sin() * mscale).to(x.dtype)
    t, rest = x[..., :rot], x[..., rot:]
    if layout == HALF:
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([t, rest], -1)


def _put(cache, rows, slots):
    """Rows [kv_heads, m, row] to the cache rows slots[m]; a slot of -1 is
    skipped (its token repeats the write of the first used one)."""
    used = slots >= 0
    at = torch.where(used, torch.arange(slots.numel(), device=slots.device), used.int().argmax())
    slot = slots[at].long()
    cache[slot // cache.shape[2], :, slot % cache.shape[2]] = rows[:, at].transpose(0, 1)


def _get(cache, slots):
    """Cache rows slots[n] as [kv_heads, n, D] in fp16; a slot of -1 gives zeros."""
    slot = slots.clamp(min=0).long()
    rows = _unpack(cache[slot // cache.shape[2], :, slot % cache.shape[2]].transpose(0, 1))
    return torch.where((slots >= 0)[:, None], rows, 0.0).half()


def _plain_write(s):
    out = {}
    turn = (s["pos"], s["inv"], s["rot"], s["layout"], 1.0)
    k, v = _rotate(s["k"].float(), *turn), s["v"].float()
    _put(s["kc"], k.half() if s["codec"] == F16 else _pack(k), s["slots"])
    _put(s["vc"], s["v"] if s["codec"] == F16 else _pack(v), s["slots"])
    if s["queries"]:
        out["q"] = _rotate(s["q"].float(), *turn).half()
    out["k"], out["v"] = _get(s["kc"], s["slots"]), _get(s["vc"], s["slots"])
    return out


def _ancestors(parents):
    """[batch, N, N] truth: node i sees node j (itself or an ancestor).  A
    parent of -1 is the context; lower ones mark unused nodes."""
    n = parents.shape[1]
    i = torch.arange(n, device=parents.device)
    step = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    step = (step @ step).clamp(max=1.0)   # 2, 4, ... 64 generations
    step = (step @ step).clamp(max=1.0)
    step = (step @ step).clamp(max=1.0)
    step = (step @ step).clamp(max=1.0)
    step = (step @ step).clamp(max=1.0)
    step = (step @ step).clamp(max=1.0)
    return (step > 0) & (parents >= -1)[:, :, None]


def _plain_tree(s):
    b, n, h, hk, d, c = s["batch"], s["nodes"], s["heads"], s["kv_heads"], s["dim"], s["capacity"]
    g = h // hk
    j = torch.arange(c, device="cuda")
    node = j - s["past"].long()[:, None]                                   # [b, c]
    seen = torch.gather(_ancestors(s["parents"]), 2, node.clamp(0, n - 1)[:, None, :].expand(b, n, c))
    used = (s["parents"] >= -1)[:, :, None]
    seen = torch.where(node[:, None, :] < 0, used, seen & (node < n)[:, None, :])   # [b, n, c]
    seen = seen[:, None, None].expand(b, hk, g, n, c).reshape(b, hk, g * n, c)
    q = s["q"].float().reshape(hk, g, b, n, d).permute(2, 0, 1, 3, 4).reshape(b, hk, g * n, d)
    score = torch.where(seen, q @ _unpack(s["kc"]).transpose(2, 3) * d ** -0.5, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = (p @ _unpack(s["vc"])) / torch.where(total > 0, total, 1.0)
    return o.reshape(b, hk, g, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, h * d).half()


def _plain_norm(s):
    u, r = s["h"].float(), s["r"].float()
    if s["post"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"].float()
    if s["g"] is not None:
        u = u * s["g"].float()
    r = s["res_scale"] * r + s["branch_scale"] * u
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["w_pre"].float()
    return {"y": y.half(), "r": r.to(s["r"].dtype)}


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s)
    if op == "rope":
        return _rotate(s["x"].float(), s["pos"], s["inv"], s["rot"], s["layout"], s["mscale"]).half()
    if op == "write":
        return _plain_write(s)
    if op == "read":
        return {"k": _get(s["kc"], s["slots"]), "v": _get(s["vc"], s["slots"])}
    if op == "tree":
        return _plain_tree(s)
    return _plain_norm(s)


def _own(s):
    import swiglu_block_quantized_gb300 as m
    op = s["op"]
    if op == "norm":
        y, r = m.norm_residual(s["h"], s["r"], s["w_pre"], w_post=s["w_post"], gate=s["g"], res_scale=s["res_scale"],
                               branch_scale=s["branch_scale"], eps=1e-6)
        return {"y": y, "r": r}
    layout = m.ROPE_HALF if s.get("layout") == HALF else m.ROPE_INTERLEAVED
    if op == "rope":
        return m.rope(s["x"], s["pos"], s["freqs"], layout=layout, mscale=s["mscale"])
    codec = m.KV_F16 if s["codec"] == F16 else m.Q8_0
    if op == "tree":
        return m.attention_tree(s["q"], s["kc"], s["vc"], codec, s["past"], s["parents"])
    out = {}
    if op == "write":
        q = m.kv_write(s["k"], s["v"], s["kc"], s["vc"], codec, s["slots"], pos=s["pos"], freqs=s["freqs"],
                       layout=layout, q=s["q"] if s["queries"] else None)
        if s["queries"]:
            out["q"] = q
    out["k"], out["v"] = m.kv_read(s["kc"], s["vc"], codec, s["slots"])
    return out


# ---------------------------------------------------------------- bytes and operations

def _row(case):
    return 2 * case["dim"] if case["codec"] == F16 else case["dim"] // 32 * 34


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["heads"] * case["rows"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    if op == "write":
        n = case["kv_heads"] * case["batch"] * case["each"]
        q = case["group"] * n * case["dim"] * 4 if case["queries"] else 0
        # K and V in, their cache rows out, and the rows read back
        return {"bytes": 2 * n * (2 * case["dim"] + 2 * _row(case) + 2 * case["dim"]) + q,
                "flops": n * (3 * case["rot"] + 6 * case["dim"])}
    if op == "read":
        n = 2 * case["kv_heads"] * case["rows"]
        return {"bytes": n * (_row(case) + 2 * case["dim"]), "flops": n * case["dim"]}
    if op == "tree":
        pasts, counts = _pasts(case), _counts(case)
        rows = 2 * case["kv_heads"] * sum(p + c for p, c in zip(pasts, counts))
        io = 4 * case["heads"] * sum(counts) * case["dim"]
        pairs = sum(c * (p + 1) for p, c in zip(pasts, counts))
        return {"bytes": rows * _row(case) + io, "flops": 4 * case["heads"] * case["dim"] * pairs}
    n = case["rows"] * case["dim"]
    each = 2 + 2 + (8 if case["res32"] else 4) + (2 if case["gate"] == "row" else 0)
    return {"bytes": n * each, "flops": 10 * n}


# ---------------------------------------------------------------- 64 bits

def _e_turn(x, s, mscale=1.0):
    theta = torch.outer(s["pos"].to(torch.float64), s["inv"])
    z = torch.polar(torch.full_like(theta, mscale), theta)
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


def _e_values(cache, codec):
    if codec == F16:
        return cache.to(torch.float64)
    b = cache.unflatten(-1, (-1, 34))
    d = (b[..., 0].to(torch.int32) + 256 * b[..., 1].to(torch.int32)).to(torch.int16).view(torch.float16)
    q = b[..., 2:].to(torch.int32)
    q = torch.where(q > 127, q - 256, q).to(torch.float64)
    return (q * d.to(torch.float64)[..., None]).to(torch.float16).to(torch.float64).flatten(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        return _e_turn(s["x"], s, s["mscale"])
    if op == "write":
        used = (s["slots"] >= 0).to(torch.float64)[:, None]
        out = {"q": _e_turn(s["q"], s)} if s["queries"] else {}
        out["k"] = _e_stored(_e_turn(s["k"], s), s["codec"]) * used
        out["v"] = _e_stored(s["v"].to(torch.float64), s["codec"]) * used
        return out
    if op == "read":
        slot = s["slots"].long()
        out = {}
        for name, cache in (("k", s["kc"]), ("v", s["vc"])):
            flat = cache.transpose(0, 1).flatten(1, 2)          # [kv_heads, batch * capacity, row]
            out[name] = _e_values(flat[:, slot], s["codec"])
        return out
    if op == "tree":
        return _e_tree(case, s)
    h, r = s["h"].to(torch.float64), s["r"].to(torch.float64)
    if s["post"]:
        h = h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * s["w_post"].to(torch.float64)
    if s["g"] is not None:
        h = h * s["g"].to(torch.float64)
    r = s["res_scale"] * r + s["branch_scale"] * h
    return {"y": r / (r.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * s["w_pre"].to(torch.float64), "r": r}


def _e_tree(case, s):
    n, h, hk, d = case["nodes"], case["heads"], case["kv_heads"], case["dim"]
    parents = s["parents"].cpu().tolist()
    out = torch.zeros(case["batch"], n, h, d, dtype=torch.float64, device="cuda")
    for b, past in enumerate(_pasts(case)):
        k = _e_values(s["kc"][b, :, :past + n], case["codec"]).repeat_interleave(h // hk, 0)
        v = _e_values(s["vc"][b, :, :past + n], case["codec"]).repeat_interleave(h // hk, 0)
        see = torch.zeros(n, past + n, dtype=torch.bool)
        for i in range(n):
            if parents[b][i] < -1:
                continue
            see[i, :past] = True
            j = i
            while j >= 0:
                see[i, past + j] = True
                j = parents[b][j]
        q = s["q"][:, b * n:(b + 1) * n].to(torch.float64)
        a = torch.einsum("hnd,hjd->hnj", q, k) / math.sqrt(d)
        a = a.masked_fill(~see.cuda(), -math.inf)
        o = torch.einsum("hnj,hjd->nhd", torch.nan_to_num(torch.softmax(a, -1)), v)
        out[b] = torch.where(see.any(1).cuda()[:, None, None], o, 0.0)
    return out.reshape(case["batch"] * n, h * d)
