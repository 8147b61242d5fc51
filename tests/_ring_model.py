"""A model of the barriers of the tree attention kernels (csrc/attention_few.cu,
csrc/attention_tree.cu), run in orders that a GPU may take and seldom does.

Every warp (two stand for four of a group) and every issuing or copying lane is
a generator that waits on mbarriers, copies land and MMAs complete when the
scheduler says so, and one of them at a time is held back until nothing else can
move.  A wait passes by the parity rule of an mbarrier; it is an error if the
phase that it was meant for is not complete (an alias), if an operand stage or
what the warps hand each other (Q, O, P, maxima, sums, ancestor bits, noted rows)
is not that of the tile or run it is read for, or if nothing can move."""
import random

W = 2   # warps that stand for a group of four


class Fault(AssertionError):
    pass


class Bar:
    def __init__(self, name, count=1):
        self.name, self.count, self.left, self.done = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.done += 1
            self.left = self.count

    def passes(self, parity):   # the phase before the current one has this parity
        return (self.done & 1) != (parity & 1)


class Sim:
    def __init__(self, seed, held):
        self.rng, self.held = random.Random(seed), held
        self.roles, self.events, self.syncs = {}, {}, {}

    def role(self, name, gen):
        self.roles[name] = [gen, next(gen, None)]

    # an event that happens at any later time; those of one queue in order
    def later(self, queue, name, act):
        self.events.setdefault(queue, []).append((name, act))

    def ready(self, name):
        op = self.roles[name][1]
        if op is None:
            return False
        if op[0] == "wait":
            return op[1].passes(op[2])
        if op[0] == "sync":
            return op[3] <= self.syncs[op[1]][1]
        return True

    def advance(self, name):
        r = self.roles[name]
        op = r[1]
        if op is not None and op[0] == "wait" and op[1].done <= op[3]:
            raise Fault("%s waited on %s for phase %d and went on with %d complete" % (name, op[1].name, op[3], op[1].done))
        r[1] = next(r[0], None)
        while r[1] is not None and r[1][0] == "sync" and len(r[1]) == 3:   # arrive at a named barrier
            key, n = r[1][1], r[1][2]
            s = self.syncs.setdefault(key, [0, 0])
            s[0] += 1
            r[1] = ("sync", key, n, (s[0] - 1) // n + 1)
            s[1] = s[0] // n

    def run(self):
        for name in list(self.roles):   # a role may begin with a named barrier
            op = self.roles[name][1]
            assert op is None or op[0] != "sync"
        while True:
            can = [("role", n) for n in self.roles if self.ready(n)]
            can += [("event", q) for q, e in self.events.items() if e]
            if not can:
                break
            free = [c for c in can if not self.is_held(c)]
            kind, key = self.rng.choice(free or can)
            if kind == "role":
                self.advance(key)
            else:
                name, act = self.events[key].pop(0)
                act()
        stuck = [n for n in self.roles if self.roles[n][1] is not None]
        if stuck:
            raise Fault("nothing moves: %s" % ", ".join("%s at %s" % (n, self.roles[n][1][1:3]) for n in stuck))

    def is_held(self, c):
        name = c[1] if c[0] == "role" else self.events[c[1]][0][0]
        return name == self.held


def wait(bar, phase):
    return ("wait", bar, phase & 1, phase)


STEP = ("step",)


class Ring:
    def __init__(self, n, name, count=1):
        self.bars = [Bar("%s[%d]" % (name, i), count) for i in range(n)]
        self.n = n

    def __getitem__(self, i):
        return self.bars[i]


class Uses:
    """Which use of its barrier a tile's landing is: the phase a wait for it means."""

    def __init__(self):
        self.count, self.of = {}, {}

    def add(self, key, tile):
        self.of[key, tile] = self.count.get(key, 0)
        self.count[key] = self.of[key, tile] + 1

    def __call__(self, key, tile):
        return self.of[key, tile]


def tiles_of(runs):
    """(run, first of it, masked) of every tile of a CTA; runs: (tiles, masked)."""
    return [(w, i == 0, i >= n - mk) for w, (n, mk) in enumerate(runs) for i in range(n)]


def few(geo, q8, runs, seed, held):
    """few_kernel: geo = ks, vs, rs, groups and raw_bar[kind][slot], the landing
    barrier of a K or V tile in a raw slot (csrc/tree_rings.h)."""
    ks_n, vs_n, rs_n, pg = geo["ks"], geo["vs"], geo["rs"], geo["groups"]
    sim = Sim(seed, held)
    tiles = tiles_of(runs)
    prep_w = 2 * pg * W if q8 else W
    noters = range(pg * W, prep_w) if q8 else range(prep_w)
    k_full, k_empty = Ring(ks_n, "k_full", W if q8 else 1), Ring(ks_n, "k_empty")
    v_full, v_empty = Ring(vs_n, "v_full", W if q8 else 1), Ring(vs_n, "v_empty")
    v_raw, v_clean = Ring(vs_n, "v_raw"), Ring(vs_n, "v_clean", prep_w)
    r_full, r_empty = Ring(2 * rs_n, "r_full"), Ring(rs_n, "r_empty", W)
    s_full, s_free = Ring(4, "s_full"), Ring(4, "s_free", W)
    p_full, p_free = Ring(2, "p_full", W), Ring(2, "p_free")
    q_full, q_empty = Bar("q_full", prep_w), Bar("q_empty")
    o_done, o_free, ml_rdy, nf_rdy = Bar("o_done"), Bar("o_free", 2 * W), Bar("ml_rdy", 2), Bar("nf_rdy", prep_w)
    kst, vst, raw = {}, {}, {}
    held_by = {}
    q_of, o_of, o_busy, ml, noted, unused = {}, {}, {}, {}, {}, {}

    def holds(store, key, tile, what):
        if store.get(key) != tile:
            raise Fault("%s of tile %s read from %s, which holds %s" % (what, tile, key, store.get(key)))

    def raw_bar(kv, slot):
        return geo["raw_bar"][kv][slot]

    land, vmask = Uses(), Uses()
    for g, (_, _, masked) in enumerate(tiles):
        for kv in range(2):
            if q8:
                sl = (2 * g + kv) % rs_n
                land.add(raw_bar(kv, sl), (kv, g))
        vmask.add(("clean" if not q8 and masked else "full", g % vs_n), g)

    def commit(who, n, act):
        sim.later(who, "%s %s" % (who, n), act)

    def issue_s():
        yield STEP
        g = 0
        for w, (n, _) in enumerate(runs):
            yield wait(q_full, w)
            for _ in range(n):
                st, sb = g % ks_n, g & 3
                yield wait(k_full[st], g // ks_n)
                if g >= 4:
                    yield wait(s_free[sb], (g >> 2) - 1)
                holds(kst, st, g, "K")

                def done(g=g, st=st, sb=sb, w=w):
                    holds(kst, st, g, "K")
                    for pw in range(prep_w):
                        holds(q_of, pw, w, "Q")
                    held_by["s", sb] = g
                    s_full[sb].arrive()
                    k_empty[st].arrive()
                commit("S", g, done)
                g += 1
            commit("S", "end %d" % w, q_empty.arrive)

    def issue_pv():
        yield STEP
        g = 0
        for w, (n, mk) in enumerate(runs):
            for i in range(n):
                vs, pb = g % vs_n, g & 1
                clean = not q8 and i >= n - mk
                yield wait((v_clean if clean else v_full)[vs], vmask(("clean" if clean else "full", vs), g))
                yield wait(p_full[pb], g >> 1)
                if i == 0 and w > 0:
                    yield wait(o_free, w - 1)
                holds(vst, vs, g, "V")
                holds(held_by, ("p", pb), g, "P")
                o_of[pb] = w
                o_busy[pb] = g

                def done(g=g, vs=vs, pb=pb):
                    holds(vst, vs, g, "V")
                    holds(held_by, ("p", pb), g, "P")
                    if o_busy[pb] == g:
                        o_busy[pb] = None
                    v_empty[vs].arrive()
                    p_free[pb].arrive()
                commit("PV", g, done)
                g += 1
            commit("PV", "end %d" % w, o_done.arrive)

    def copies(kinds):
        yield STEP
        n = 0
        for g, (_, _, masked) in enumerate(tiles):
            for kv in kinds:
                if q8:
                    sl = n % rs_n
                    if n >= rs_n:
                        yield wait(r_empty[sl], n // rs_n - 1)

                    def lands(sl=sl, kv=kv, g=g):
                        raw[sl] = (kv, g)
                        r_full[raw_bar(kv, sl)].arrive()
                else:
                    sl = n % (vs_n if kv else ks_n)
                    if n >= (vs_n if kv else ks_n):
                        yield wait((v_empty if kv else k_empty)[sl], n // (vs_n if kv else ks_n) - 1)

                    def lands(sl=sl, kv=kv, g=g, masked=masked):
                        (vst if kv else kst)[sl] = g
                        ((v_raw if masked else v_full) if kv else k_full)[sl].arrive()
                sim.later(("copy", kv, g), "copy %d %d" % (kv, g), lands)
                n += 1

    def softmax(team, sw):
        yield STEP
        g = 0
        for w, (n, mk) in enumerate(runs):
            if mk and team == 0 and sw == 0:
                unused[w & 1] = w
            for i in range(n):
                if (g & 1) == team:
                    sb = g & 3
                    yield wait(s_full[sb], g >> 2)
                    if g >= 2:
                        yield wait(p_free[team], (g >> 1) - 1)
                    holds(held_by, ("s", sb), g, "S")
                    s_free[sb].arrive()
                    yield ("sync", "team %d" % team, W)
                    if i >= 2:   # O rescaled
                        holds(o_busy, team, None, "O")
                        holds(o_of, team, w, "O")
                    yield STEP
                    held_by["p", team] = g
                    p_full[team].arrive()
                g += 1
            yield ("sync", "team %d" % team, W)
            yield STEP
            if sw == 0:
                ml[w & 1, team] = w
                ml_rdy.arrive()
            yield wait(ml_rdy, w)
            yield wait(o_done, w)
            yield wait(nf_rdy, w)
            yield ("sync", "team %d" % team, W)
            yield STEP
            for t in range(2):
                holds(ml, (w & 1, t), w, "(m, l)")
                if any((x & 1) == t for x in range(g - n, g)):
                    holds(o_busy, t, None, "O")
                    holds(o_of, t, w, "O")
            if mk:
                holds(unused, w & 1, w, "unused rows")
                for pw in noters:
                    holds(noted, (w & 1, pw), w, "noted rows")
            o_free.arrive()

    def prepare(pw):
        kv, turn = (pw // (W * pg), (pw // W) % pg) if q8 else (1, 0)
        raw_waits = {}
        yield STEP
        g = 0
        for w, (n, mk) in enumerate(runs):
            if w > 0:
                yield wait(q_empty, w - 1)
            noted[w & 1, pw] = w
            q_of[pw] = w
            yield STEP
            q_full.arrive()
            for i in range(n):
                ks, vs = g % ks_n, g % vs_n
                if q8:
                    rs = (2 * g + kv) % rs_n
                    if pg == 1 or (g & 1) == turn:
                        if g >= (vs_n if kv else ks_n):
                            yield wait(v_empty[vs] if kv else k_empty[ks], g // (vs_n if kv else ks_n) - 1)
                        yield wait(r_full[raw_bar(kv, rs)], land(raw_bar(kv, rs), (kv, g)))
                        holds(raw, rs, (kv, g), "raw")
                        yield STEP
                        holds(raw, rs, (kv, g), "raw")
                        (vst if kv else kst)[vs if kv else ks] = g
                        r_empty[rs].arrive()
                        yield STEP
                        (v_full[vs] if kv else k_full[ks]).arrive()
                elif i >= n - mk:
                    raw_waits[vs] = raw_waits.get(vs, -1) + 1
                    yield wait(v_raw[vs], raw_waits[vs])
                    holds(vst, vs, g, "V to clear")
                    v_clean[vs].arrive()
                g += 1
            if w >= 1:
                yield wait(o_free, w - 1)
            nf_rdy.arrive()

    sim.role("S issuer", issue_s())
    sim.role("PV issuer", issue_pv())
    if q8:
        sim.role("copies", copies((0, 1)))
    else:
        sim.role("K copies", copies((0,)))
        sim.role("V copies", copies((1,)))
    for team in range(2):
        for sw in range(W):
            sim.role("softmax %d.%d" % (team, sw), softmax(team, sw))
    for pw in range(prep_w):
        sim.role("prepare %d" % pw, prepare(pw))
    sim.run()


FEW_ROLES = ["S issuer", "PV issuer", "copies", "K copies", "V copies", "softmax 0.0", "softmax 1.1", "prepare 0",
             "prepare 1", "prepare %d" % W, "prepare %d" % (2 * W), "prepare %d" % (3 * W)]


def rows(geo, q8, runs, seed, held):
    """tree_kernel: geo = ks, vs, rs, sb (score buffers), k_bar[team][stage], the
    landing barrier of a K stage, and max_slot[g % 4], where the halves of a row
    exchange the maxima of tile g (csrc/tree_rings.h)."""
    ks_n, vs_n, rs_n, sb_n = geo["ks"], geo["vs"], geo["rs"], geo["sb"]
    sim = Sim(seed, held)
    tiles = tiles_of(runs)
    quads = (0, 1)                      # two stand for four; the second has rows in odd seeds
    parts = [(quad, half) for quad in quads[:1 + seed % 2] for half in range(2)]   # of a score buffer
    soft = 2 * 2 * len(quads)           # teams, halves
    prep_w = 2 * W if q8 else W
    noters = range(W, prep_w) if q8 else range(prep_w)
    k_full, k_empty = Ring(2 * ks_n, "k_full", W if q8 else 1), Ring(ks_n, "k_empty")
    v_full, v_empty = Ring(vs_n, "v_full", W if q8 else 1), Ring(vs_n, "v_empty")
    v_raw, v_clean = Ring(vs_n, "v_raw"), Ring(vs_n, "v_clean", prep_w)
    r_full, r_empty = Ring(2 * rs_n, "r_full"), Ring(rs_n, "r_empty", W)
    s_full, p_full = Ring(4, "s_full"), Ring(4, "p_full", 2 * len(quads))
    pv_done = Ring(sb_n, "pv_done")
    q_full, q_empty = Bar("q_full", prep_w), Bar("q_empty", 2)
    ml_rdy, nf_rdy, o_free = Bar("ml_rdy", 2 * len(quads)), Bar("nf_rdy", prep_w), Bar("o_free", soft)
    kst, vst, raw, buf, maxima = {}, {}, {}, {}, {}
    q_of, o_of, o_busy, ml, sums, noted, bits, up = {}, {}, {}, {}, {}, {}, {}, {}

    def holds(store, key, tile, what):
        if store.get(key) != tile:
            raise Fault("%s of tile %s read from %s, which holds %s" % (what, tile, key, store.get(key)))

    k_land, r_land, v_land, team_use = Uses(), Uses(), Uses(), Uses()
    for g, (_, _, masked) in enumerate(tiles):
        k_land.add(geo["k_bar"][g & 1][g % ks_n], g)
        v_land.add(("clean" if not q8 and masked else "full", g % vs_n), g)
        team_use.add(2 * (g & 1) + ((g >> 1) & 1), g)
        for kv in range(2):
            if q8:
                r_land.add((kv, (2 * g + kv) % rs_n), g)

    def sp_of(g):
        return 2 * (g & 1) + ((g >> 1) & 1)

    def issue(team):
        yield STEP
        g = 0
        who = "S%d" % team

        def pv_wait(x):
            if x >= 0:
                yield wait(pv_done[x % sb_n], x // sb_n)

        def scores(x, w):
            st = x % ks_n
            yield wait(k_full[geo["k_bar"][team][st]], k_land(geo["k_bar"][team][st], x))
            holds(kst, st, x, "K")

            def done():
                holds(kst, st, x, "K")
                for pw in range(prep_w):
                    holds(q_of, pw, w, "Q")
                for part in parts:
                    buf[x % sb_n, part] = ("s", x)
                s_full[sp_of(x)].arrive()
                k_empty[st].arrive()
            sim.later(who, "%s %d" % (who, x), done)

        for w, (n, mk) in enumerate(runs):
            mine = [(x, x - g >= n - mk) for x in range(g, g + n) if (x & 1) == team]
            g += n
            yield wait(q_full, w)
            if not mine:
                sim.later(who, "%s q %d" % (who, w), q_empty.arrive)
                continue
            if sb_n == 3:
                yield from pv_wait(mine[0][0] - 3)
                yield from scores(mine[0][0], w)
            for i, (x, masked) in enumerate(mine):
                more = i + 1 < len(mine)
                if sb_n == 2:
                    yield from pv_wait(x - 2)
                    yield from scores(x, w)
                else:
                    yield from pv_wait(x - 1)
                    if more:
                        yield from scores(mine[i + 1][0], w)
                if not more:
                    sim.later(who, "%s q %d" % (who, w), q_empty.arrive)
                vs = x % vs_n
                clean = not q8 and masked
                yield wait((v_clean if clean else v_full)[vs], v_land(("clean" if clean else "full", vs), x))
                if i == 0 and w > 0:
                    yield wait(o_free, w - 1)
                yield wait(p_full[sp_of(x)], team_use(sp_of(x), x))
                holds(vst, vs, x, "V")
                for part in parts:
                    holds(buf, (x % sb_n, part), ("p", x), "P")
                o_of[team] = w
                o_busy[team] = x

                def done(x=x, vs=vs):
                    o_busy[team] = None
                    holds(vst, vs, x, "V")
                    for part in parts:
                        holds(buf, (x % sb_n, part), ("p", x), "P")
                    pv_done[x % sb_n].arrive()
                    v_empty[vs].arrive()
                sim.later(who, "%s PV %d" % (who, x), done)

    def copies(kinds):
        yield STEP
        n = 0
        for g, (_, _, masked) in enumerate(tiles):
            for kv in kinds:
                if q8:
                    sl = n % rs_n
                    if n >= rs_n:
                        yield wait(r_empty[sl], n // rs_n - 1)

                    def lands(sl=sl, kv=kv, g=g):
                        raw[sl] = (kv, g)
                        r_full[kv * rs_n + sl].arrive()
                else:
                    size = vs_n if kv else ks_n
                    sl = n % size
                    if n >= size:
                        yield wait((v_empty if kv else k_empty)[sl], n // size - 1)

                    def lands(sl=sl, kv=kv, g=g, masked=masked):
                        (vst if kv else kst)[sl] = g
                        if kv:
                            (v_raw if masked else v_full)[sl].arrive()
                        else:
                            k_full[geo["k_bar"][g & 1][sl]].arrive()
                sim.later(("copy", kv, g), "copy %d %d" % (kv, g), lands)
                n += 1

    def softmax(team, half, quad):
        busy = quad <= seed % 2
        pair, whole = "pair %d %d" % (team, quad), "quad %d" % quad
        yield STEP
        g = 0
        for w, (n, mk) in enumerate(runs):
            if busy and mk:
                yield ("sync", whole, 4)
                yield STEP
                if team == 0 and not half:
                    up["tree"] = w
                    yield STEP
                    holds(up, "tree", w, "parents")
                    bits[quad] = w
                yield ("sync", whole, 4)
                yield STEP
                holds(bits, quad, w, "ancestor bits")
            for i in range(n):
                x, g = g, g + 1
                if (x & 1) != team:
                    continue
                sp = sp_of(x)
                yield wait(s_full[sp], team_use(sp, x))
                if not busy:
                    p_full[sp].arrive()
                    continue
                holds(buf, (x % sb_n, (quad, half)), ("s", x), "S")
                slot = geo["max_slot"][x % 4]
                maxima[slot, team, half] = x
                yield ("sync", pair, 2)
                yield STEP
                holds(maxima, (slot, team, 1 - half), x, "maximum")
                if sb_n == 3 and i >= 2 and sim.rng.random() < 0.5:   # references rise
                    yield wait(pv_done[(x - 2) % sb_n], (x - 2) // sb_n)
                    holds(o_busy, team, None, "O")
                    holds(o_of, team, w, "O")
                elif sb_n == 2 and i >= 2:
                    holds(o_busy, team, None, "O")
                    holds(o_of, team, w, "O")
                yield STEP
                if mk:
                    holds(bits, quad, w, "ancestor bits")
                holds(buf, (x % sb_n, (quad, half)), ("s", x), "S")
                buf[x % sb_n, (quad, half)] = ("p", x)
                p_full[sp].arrive()
            if half:
                sums[team, quad] = w
            yield ("sync", pair, 2)
            yield STEP
            if not half:
                holds(sums, (team, quad), w, "sums")
                ml[w & 1, team, quad] = w
                ml_rdy.arrive()
            yield wait(ml_rdy, w)
            yield wait(nf_rdy, w)
            yield wait(pv_done[(g - 1) % sb_n], (g - 1) // sb_n)
            if sb_n == 2 and g > 1:
                yield wait(pv_done[(g - 2) % sb_n], (g - 2) // sb_n)
            yield ("sync", whole, 4)
            yield STEP
            for t in range(2):
                holds(ml, (w & 1, t, quad), w, "(m, l)")
                if any((x & 1) == t for x in range(g - n, g)):
                    holds(o_busy, t, None, "O")
                    holds(o_of, t, w, "O")
            if busy and mk:
                holds(bits, quad, w, "ancestor bits")
                for pw in noters:
                    holds(noted, (w & 1, pw), w, "noted rows")
            o_free.arrive()

    def prepare(pw):
        kv = pw // W
        raw_waits = {}
        yield STEP
        g = 0
        for w, (n, mk) in enumerate(runs):
            if w > 0:
                yield wait(q_empty, w - 1)
            noted[w & 1, pw] = w
            q_of[pw] = w
            yield STEP
            q_full.arrive()
            for i in range(n):
                ks, vs = g % ks_n, g % vs_n
                if q8:
                    rs = (2 * g + kv) % rs_n
                    yield wait(r_full[kv * rs_n + rs], r_land((kv, rs), g))
                    st, size = (vs, vs_n) if kv else (ks, ks_n)
                    if g >= size:
                        yield wait((v_empty if kv else k_empty)[st], g // size - 1)
                    holds(raw, rs, (kv, g), "raw")
                    yield STEP
                    holds(raw, rs, (kv, g), "raw")
                    (vst if kv else kst)[st] = g
                    (v_full[st] if kv else k_full[geo["k_bar"][g & 1][st]]).arrive()
                    yield STEP
                    r_empty[rs].arrive()
                elif i >= n - mk:
                    raw_waits[vs] = raw_waits.get(vs, -1) + 1
                    yield wait(v_raw[vs], raw_waits[vs])
                    holds(vst, vs, g, "V to clear")
                    v_clean[vs].arrive()
                g += 1
            if w >= 1:
                yield wait(o_free, w - 1)
            nf_rdy.arrive()

    for team in range(2):
        sim.role("issuer %d" % team, issue(team))
        for half in range(2):
            for quad in quads:
                sim.role("softmax %d.%d.%d" % (team, half, quad), softmax(team, half, quad))
    if q8:
        sim.role("copies", copies((0, 1)))
    else:
        sim.role("K copies", copies((0,)))
        sim.role("V copies", copies((1,)))
    for pw in range(prep_w):
        sim.role("prepare %d" % pw, prepare(pw))
    sim.run()


ROWS_ROLES = ["issuer 0", "issuer 1", "copies", "K copies", "V copies", "softmax 0.0.0", "softmax 0.1.0", "softmax 1.0.0",
              "softmax 1.1.0", "softmax 0.0.1", "softmax 1.1.1", "prepare 0", "prepare 1", "prepare %d" % W]


def held_things(tiles, roles):
    """What is held back, one at a time: each role, each of a few copies and MMAs."""
    copies = ["copy %d %d" % (kv, g) for g in range(min(tiles, 9)) for kv in range(2)]
    return [None] + roles + copies + \
        ["%s %d" % (q, g) for q in ("S", "PV", "S0", "S1", "S0 PV", "S1 PV") for g in range(min(tiles, 6))]
