"""A CPU model of the paged attention kernel's barrier protocol.

attn_paged_kernel (csrc/attn_paged.cu) walks a span of segments with seven
roles: a K producer that also publishes the segments' descriptors and copies
Q, a V producer, two MMA issuers and two softmax groups (one role each here).
Their waits test a barrier's phase parity, so a waiter must never fall two
phases behind: it would block, or pass on the wrong phase. Device waits are
bounded, so a fault of the protocol would show as a timeout status or, worse,
as a silent race; this model finds both on the CPU.

Each role is a generator that yields the barrier phase it waits for. Copies
land in any order at random times, and the tensor pipe runs MMAs and commits in
order at random times. Every wait and every test checks that the barrier is at
the awaited phase or one past it, and every access checks what it finds: the
ring's slots, the Q tiles, S / P and O of each group, the descriptors. Planted
mistakes must be caught.
"""

import random

import pytest

SEGS, PAIR, SPLIT, SOLO0, SOLO1 = 4, 0, 1, 2, 3


class _Fault(Exception):
    pass


def _check(cond, what):
    if not cond:
        raise _Fault(what)


class _Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def done(self, idx):
        """Whether phase idx is complete, as a parity test can tell."""
        _check(idx <= self.phase <= idx + 1, "phase %d, waiter wants %d" % (self.phase, idx))
        return self.phase == idx + 1


def segment(rng, last, solo, q, longest=9):
    """A random segment as Span::next hands it out; q, solo: the ring numbers so far."""
    pair = rng.random() < 0.35
    length = rng.choice([0, 1, 1, 2, 3, 4, 5, rng.randint(1, longest)])
    kb = rng.choice([0, 0, 3])
    s = dict(kb=kb, ke=kb + length, q=q)
    if pair:
        s.update(mode=PAIR, n=(rng.choice([length, max(0, length - 1), rng.randint(0, length)]), length))
        q += 2 if length else 0
    else:
        if length > 4 or last:
            s.update(mode=SPLIT, n=((length + 1) // 2, length // 2))
        else:
            t = solo & 1
            solo += 1
            s.update(mode=SOLO0 + t, n=(length if t == 0 else 0, length if t == 1 else 0))
        q += 1 if length else 0
    return s, solo, q


def span(rng, count):
    out, solo, q = [], 0, 0
    for i in range(count):
        s, solo, q = segment(rng, i + 1 == count, solo, q)
        out.append(s)
    return out


def _needs(s, t, u):
    if s["mode"] == PAIR:
        return u < s["kb"] + s["n"][t]
    if s["mode"] == SPLIT:
        return (u - s["kb"]) & 1 == t
    return s["n"][t] > 0


def _tiles(s):
    return 2 if s["mode"] == PAIR else 1


def _run(segs, rings, rng, planted=None, p_resc=0.3):
    """True when every role finishes; raises _Fault on a hazard; False on deadlock.
    rings: the slots of K and of V."""
    NK, NV = rings
    NS = NK + NV
    end = len(segs)

    # (slot, use) of a step's K and V tiles; n: the steps before it
    def slot_k(n):
        return (2 * n % NS, 2 * n // NS) if planted == "one_ring" else (n % NK, n // NK)

    def slot_v(n):
        return ((2 * n + 1) % NS, (2 * n + 1) // NS) if planted == "one_ring" else \
            (NK + n % NV, n // NV)

    B = {"split_ready": _Bar(1), "split_read": _Bar(1)}
    for i in range(SEGS):
        B["seg_full", i], B["seg_empty", i] = _Bar(1), _Bar(5)
    for i in range(NS):
        B["kv_full", i], B["kv_empty", i] = _Bar(1), _Bar(2)
    for t in range(2):
        B["q_full", t], B["q_empty", t] = _Bar(1), _Bar(2)
        B["s_full", t], B["o_done", t], B["group", t] = _Bar(1), _Bar(1), _Bar(2)
    seg_slot = [None] * SEGS
    kv, qs = [None] * NS, [None] * 2        # landed contents
    S, O = [None, None], [None, None]
    o_read = [-1, -1]                       # last segment whose O the epilogue has read
    reads = {}                              # content -> groups whose MMA has read it
    tma, pipe = [], []

    def wait(name, idx):
        return (name, idx)

    def seg(k):
        _check(seg_slot[k % SEGS] == k, "descriptor %d holds %r" % (k, seg_slot[k % SEGS]))
        return segs[k] if k < end else None

    def copy(where, i, tag):
        old = where[i]
        if old is not None:
            _check(old[0] != "landing", "copy into a slot that another copy is on its way to")
            kind, k, x = old
            s = segs[k]
            want = {t for t in range(2)
                    if (_needs(s, t, x) if kind != "Q" else
                        s["n"][t] > 0 and (_tiles(s) == 1 or x == t))}
            _check(reads.get(old, set()) == want, "copy over %r, read by %r of %r"
                   % (old, reads.get(old), want))
        where[i] = ("landing",)
        tma.append((where, i, tag, ("kv_full" if where is kv else "q_full", i)))

    def publish(k):
        if k >= SEGS:
            yield wait(("seg_empty", k % SEGS), k // SEGS - 1)
        seg_slot[k % SEGS] = k
        B["seg_full", k % SEGS].arrive()

    def k_producer():
        n = 0
        yield from publish(0)
        for k, s in enumerate(segs):
            yield from publish(k + 1)
            q_due = s["ke"] > s["kb"]
            for u in range(s["kb"], s["ke"]):
                slot, use = slot_k(n)
                if use > 0:
                    yield wait(("kv_empty", slot), use - 1)
                copy(kv, slot, ("K", k, u))
                if q_due:
                    lq = s["q"] + _tiles(s) - 1
                    must = u > s["kb"] or u + 1 == s["ke"]
                    if must or lq < 2 or B["q_empty", lq & 1].done((lq >> 1) - 1):
                        for i in range(_tiles(s)):
                            x = s["q"] + i
                            if x >= 2 and planted != "q_early":
                                yield wait(("q_empty", x & 1), (x >> 1) - 1)
                            copy(qs, x & 1, ("Q", k, i))
                        q_due = False
                n += 1

    def v_producer():
        n = 0
        for k in range(end + 1):
            yield wait(("seg_full", k % SEGS), k // SEGS)
            s = seg(k)
            B["seg_empty", k % SEGS].arrive()
            if s is None:
                return
            for u in range(s["kb"], s["ke"]):
                slot, use = slot_v(n)
                if use > 0:
                    yield wait(("kv_empty", slot), use - 1)
                copy(kv, slot, ("V", k, u))
                n += 1

    def issuer(t):
        st = dict(n=0, v=0, started=-1, n_seg=0, n_iss=0, seg=None, u=0, q=0)
        groups = 0

        def advance():
            """-> the group's next step, None at the segment's end"""
            a = st["seg"]
            while a is not None and st["u"] < a["ke"]:
                u, n = st["u"], st["n"]
                st["u"] += 1
                st["n"] += 1
                if _needs(a, t, u):
                    return n
                for slot, use in (slot_k(n), slot_v(n)):
                    yield wait(("kv_full", slot), use)
                    if planted != "no_release":
                        B["kv_empty", slot].arrive()
            return None

        def next_k():
            n = yield from advance()
            if n is not None:
                slot, use = slot_k(n)
                yield wait(("kv_full", slot), use)
            return n

        def try_k():
            a = st["seg"]
            while st["u"] < a["ke"]:
                n, mine = st["n"], _needs(a, t, st["u"])
                k, v = slot_k(n), slot_v(n)
                if not B["kv_full", k[0]].done(k[1]):
                    return None
                if not mine:
                    if not B["kv_full", v[0]].done(v[1]):
                        return None
                    B["kv_empty", k[0]].arrive()
                    B["kv_empty", v[0]].arrive()
                st["n"] += 1
                st["u"] += 1
                if mine:
                    return n
            return None

        def qk(n):
            k, jj = st["started"], st["n_iss"]
            pipe.append(("qk", t, k, jj, slot_k(n)[0], st["q"]))
            pipe.append(("commit", ("s_full", t)))
            pipe.append(("commit", ("kv_empty", slot_k(n)[0])))
            st["n_iss"] += 1
            if st["n_iss"] == st["n_seg"]:
                pipe.append(("commit", ("q_empty", st["q"])))
            st["v"] = n

        def start(k):
            st.update(started=k, n_seg=0, n_iss=0)
            yield wait(("seg_full", k % SEGS), k // SEGS)
            a = seg(k)
            if a is None or a["kb"] == a["ke"]:
                return
            st.update(seg=a, u=a["kb"], n_seg=a["n"][t])
            for i in range(_tiles(a)):
                x = a["q"] + i
                yield wait(("q_full", x & 1), x >> 1)
                if st["n_seg"] > 0 and (_tiles(a) == 1 or i == t):
                    st["q"] = x & 1
                else:
                    B["q_empty", x & 1].arrive()
            if st["n_seg"] == 0:
                yield from advance()
                return
            n = yield from next_k()
            if n is not None:
                qk(n)

        for k in range(end + 1):
            yield wait(("seg_full", k % SEGS), k // SEGS)
            s = seg(k)
            if s is not None and st["started"] < k:
                yield from start(k)
            B["seg_empty", k % SEGS].arrive()
            if s is None:
                B["group", t].arrive()
                yield wait(("group", t), groups)
                return
            if s["mode"] >= SOLO0 and s["mode"] != SOLO0 + t:
                continue
            n = s["n"][t]
            for jj in range(n):
                last = jj + 1 == n
                fast = None
                v, use = slot_v(st["v"])
                yield wait(("kv_full", v), use)
                if not last:
                    fast = try_k()
                B["group", t].arrive()
                yield wait(("group", t), groups)
                groups += 1
                pipe.append(("pv", t, k, jj, v))
                if fast is not None:
                    qk(fast)
                pipe.append(("commit", ("kv_empty", v)))
                if last:
                    pipe.append(("commit", ("o_done", t)))
                elif fast is None:
                    ks = yield from next_k()
                    if ks is not None:
                        qk(ks)
            if n > 0:
                yield from advance()
                yield from start(k + 1)
                if st["n_seg"] == 0 and k + 1 < end:
                    seg(k + 1)
                    yield from start(k + 2)

    def softmax(t):
        tile = groups = o_segs = n_split = 0
        for k in range(end + 1):
            yield wait(("seg_full", k % SEGS), k // SEGS)
            s = seg(k)
            B["seg_empty", k % SEGS].arrive()
            if s is None:
                B["group", t].arrive()
                yield wait(("group", t), groups)
                return
            if s["mode"] >= SOLO0 and s["mode"] != SOLO0 + t:
                continue
            n = s["n"][t]
            for jj in range(n):
                yield wait(("s_full", t), tile)
                _check(S[t] == ("S", k, jj), "scores %r" % (S[t],))
                if jj > 0 and rng.random() < p_resc:
                    _check(not any(op[0] == "pv" and op[1] == t for op in pipe),
                           "O rescaled under a running P.V")
                    _check(O[t] == (k, jj), "O rescaled: %r" % (O[t],))
                S[t] = ("P", k, jj)
                tile += 1
                B["group", t].arrive()
                yield wait(("group", t), groups)
                groups += 1
            if n > 0:
                yield wait(("o_done", t), o_segs)
                o_segs += 1
                _check(O[t] == (k, n), "epilogue before the last P.V: %r" % (O[t],))
            if s["mode"] == SPLIT and t == 1:
                B["split_ready"].arrive()
                if planted != "no_split_read":
                    yield wait("split_read", n_split)
                n_split += 1
            elif s["mode"] == SPLIT:
                yield wait("split_ready", n_split)
                n_split += 1
                _check(s["n"][1] == 0 or O[1] == (k, s["n"][1]), "group 1's O: %r" % (O[1],))
                o_read[1] = k
                o_read[0] = k
                B["split_read"].arrive()
            if s["mode"] != SPLIT:
                o_read[t] = k

    roles = {"k": k_producer(), "v": v_producer()}
    for t in range(2):
        roles["issue", t], roles["softmax", t] = issuer(t), softmax(t)
    waiting, finished = {r: None for r in roles}, set()

    def step(r):
        try:
            waiting[r] = next(roles[r])
        except StopIteration:
            finished.add(r)

    def run_pipe_head():
        op = pipe.pop(0)
        if op[0] == "commit":
            B[op[1]].arrive()
            return
        kind, t, k, jj = op[:4]
        s = segs[k]
        u = s["kb"] + (2 * jj + t if s["mode"] == SPLIT else jj)
        if kind == "qk":
            _check(kv[op[4]] == ("K", k, u), "Q K^T of %r reads %r" % ((k, u), kv[op[4]]))
            want = ("Q", k, t if s["mode"] == PAIR else 0)
            _check(qs[op[5]] == want, "Q K^T of %r reads %r" % (want, qs[op[5]]))
            _check(S[t] is None or S[t][0] == "used", "S overwritten: %r" % (S[t],))
            reads.setdefault(kv[op[4]], set()).add(t)
            if jj + 1 == s["n"][t]:
                reads.setdefault(want, set()).add(t)
            S[t] = ("S", k, jj)
        else:
            _check(kv[op[4]] == ("V", k, u), "P.V of %r reads %r" % ((k, u), kv[op[4]]))
            _check(S[t] == ("P", k, jj), "P.V before P: %r" % (S[t],))
            reads.setdefault(kv[op[4]], set()).add(t)
            if jj == 0:
                _check(O[t] is None or o_read[t] >= O[t][0], "O overwritten before its epilogue")
            else:
                _check(O[t] == (k, jj), "P.V accumulates into %r" % (O[t],))
            O[t] = (k, jj + 1)
            S[t] = ("used",)

    # one of the roles (or the copies, or the tensor pipe) is often much slower
    slow = rng.choice([None, "tma", "pipe", *roles])
    for r in roles:
        step(r)
    for _ in range(500_000):
        moves = [r for r in roles if r not in finished and B[waiting[r][0]].done(waiting[r][1])]
        moves += ["tma"] * bool(tma) + ["pipe"] * bool(pipe)
        if not moves:
            return len(finished) == len(roles)
        m = rng.choice(moves)
        if m == slow and len(moves) > 1 and rng.random() < 0.9:
            continue
        if m == "tma":
            where, i, tag, bar = tma.pop(rng.randrange(len(tma)))
            where[i] = tag
            B[bar].arrive()
        elif m == "pipe":
            run_pipe_head()
        else:
            step(m)
    raise AssertionError("the model did not terminate")


@pytest.mark.parametrize("rings", [(2, 3), (6, 6)])      # d = 128 and d = 64
@pytest.mark.parametrize("seed", range(60))
def test_protocol_completes_without_hazards(rings, seed):
    rng = random.Random(seed)
    segs = span(rng, rng.choice([1, 1, 2, 3, 6, 12, 20]))
    for run in range(4):
        assert _run(segs, rings, random.Random(1000 * seed + run), p_resc=run / 3)


@pytest.mark.parametrize("rings", [(2, 3), (6, 6)])
@pytest.mark.parametrize("segs", [
    [],                                           # a CTA without a span
    [dict(kb=0, ke=0, q=0, mode=SPLIT, n=(0, 0))],
    [dict(kb=0, ke=1, q=0, mode=SPLIT, n=(1, 0))],
    [dict(kb=0, ke=300, q=0, mode=SPLIT, n=(150, 150))],
    [dict(kb=0, ke=200, q=0, mode=PAIR, n=(199, 200))],
    [dict(kb=3, ke=9, q=0, mode=PAIR, n=(0, 6))],  # the last part of an item: tile 0 is done
])
def test_protocol_at_the_edges(rings, segs):
    for run in range(6):
        assert _run(segs, rings, random.Random(run))


@pytest.mark.parametrize("planted", ["q_early", "no_release", "no_split_read", "one_ring"])
def test_planted_mistakes_are_caught(planted):
    caught = 0
    for seed in range(60):
        rng = random.Random(seed)
        try:
            caught += not _run(span(rng, 12), (2, 3), rng, planted=planted)
        except _Fault:
            caught += 1
    assert caught > 0
