"""A CPU model of the roles of a paged-attention CTA: scheduler, producer, two MMA issuers and
two softmax streams, with their mbarriers, the ring of pieces, the K / V stages and the buffers
of Q, S, P and O, run under random schedules.

It follows the waits between the roles in csrc/paged_attn.cuh, paged_attn.cu and paged_few.cu
(those among the warps of one stream are left out).  A barrier is a
count and a phase, a wait looks at the phase's parity only (so a waiter that is two phases off
passes, as on the device), copies and tensor-core work finish in any order that the device
allows, and every buffer remembers what it holds: a role that reads something else fails an
assertion; no role able to go on is a deadlock.
"""
from __future__ import annotations

import random
from dataclasses import dataclass

RING = 8


@dataclass(frozen=True)
class Layout:
    """One of the kernels.  rings: of K / V stages (1: both issuers use every tile, two tiles of
    query rows; 2: the streams take turns); per: stages of a ring; ahead: S tiles of a stream
    ahead of its P V; buffers: of S, P and O of a stream; deferred: a unit's epilogue runs
    under the next unit's first tile."""
    rings: int
    per: int
    ahead: int
    buffers: int
    deferred: bool


LAYOUTS = {
    "few_d128": Layout(2, 3, 2, 2, True),
    "few_d64": Layout(2, 6, 2, 2, True),
    "one_tile_d128": Layout(2, 2, 1, 1, False),
    "one_tile_d64": Layout(2, 4, 1, 1, False),
    "two_tiles_d128": Layout(1, 4, 1, 1, False),
    "two_tiles_d64": Layout(1, 8, 1, 1, False),
}


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


def run(units, layout, seed, empty_in_ring=False):
    """'ok', or 'deadlock'.  units: key tiles of each unit of the CTA in order, 0 for a unit
    that sees no key; empty_in_ring: such units go through the ring too (what the scheduler
    must not do)."""
    rng = random.Random(seed)
    two = layout.rings == 1                       # both issuers use every tile
    per, ahead, nb = layout.per, layout.ahead, layout.buffers
    run_ahead = layout.rings * ahead
    pieces = [n for n in units if n or empty_in_ring]
    first = [sum(pieces[:i]) for i in range(len(pieces))]
    END = len(pieces)

    def place(t, i):
        return ((t & 1) * per if not two else 0) + i % per, i // per & 1

    def k_at(t):
        i = t if two else t >> 1
        return place(t, i if i < ahead else 2 * i - ahead + 1)

    def v_at(t):
        return place(t, 2 * (t if two else t >> 1) + ahead)

    consumers = 5                                 # producer, issuers, softmax streams
    ring_full, ring_empty = ([Barrier(c) for _ in range(RING)] for c in (1, consumers))
    q_full, q_empty = ([Barrier(c) for _ in range(2)] for c in (1, 2))
    stages = layout.rings * per
    kv_full, kv_empty = ([Barrier(c) for _ in range(stages)] for c in (1, 2 if two else 1))
    pair = lambda c: [[Barrier(c) for _ in range(nb)] for _ in range(2)]
    s_full, p_full, o_full, o_empty = pair(1), pair(1), pair(1), pair(1 if two else 2)
    meet = Barrier(2)
    ring, ring_users = [None] * RING, [0] * RING
    stage, qbuf = [None] * stages, [None, None]
    sbuf, obuf = [[None] * nb for _ in range(2)], [[None] * nb for _ in range(2)]
    copies, pipe = [], [[], []]

    def wait(bar, parity):
        return lambda: bar.passed(parity)

    def fetch(i):
        yield wait(ring_full[i % RING], i // RING)

    def release(i):
        ring_users[i % RING] -= 1
        ring_empty[i % RING].arrive()

    def scheduler():
        for i in range(END + 1):
            at = i % RING
            yield wait(ring_empty[at], i // RING ^ 1)
            assert ring_users[at] == 0, "a piece in use is overwritten"
            ring[at], ring_users[at] = i, consumers
            ring_full[at].arrive()

    def producer():
        at, j, j_end, more, new = -1, 0, 0, True, False
        tk = tv = n = pending = 0

        def advance():
            nonlocal at, j, j_end, more, new
            while more and j == j_end:
                if at >= 0:
                    release(at)
                at += 1
                yield from fetch(at)
                assert ring[at % RING] == at
                more = at < END
                j, j_end, new = 0, pieces[at] if more else 0, True
            if more:
                j += 1

        yield from advance()
        while True:
            if more:
                if new:
                    b, use = (0, n) if two else (n & 1, n >> 1)
                    yield wait(q_empty[b], use ^ 1)
                    copies.append(("q", b, at))
                    n, new = n + 1, False
                s, ph = k_at(tk)
                yield wait(kv_empty[s], ph ^ 1)
                copies.append(("kv", s, ("K", tk)))
                tk, pending = tk + 1, pending + 1
                yield from advance()
                if pending < run_ahead:
                    continue
            if pending == 0:
                return
            s, ph = v_at(tv)
            yield wait(kv_empty[s], ph ^ 1)
            copies.append(("kv", s, ("V", tv)))
            tv, pending = tv + 1, pending - 1

    def issuer(st):
        ops = pipe[st]
        step = 1 if two else 2
        S = dict(at=-1, j=0, end=0, base=0, count=0, units=0, q=0, more=True, items=0)
        at_o, j_o, end_o, base_o, count_o, items_o, sums = -1, 0, 0, 0, 0, 0, 0
        more_o = start = True

        def first_tile(count):
            return 0 if two else (count & 1) ^ st

        def prepare():
            while S["more"] and S["j"] >= S["end"]:
                S["at"] += 1
                yield from fetch(S["at"])
                S["more"] = S["at"] < END
                nt = pieces[S["at"]] if S["more"] else 0
                if not S["more"] or nt == 0:
                    continue
                S["q"] = 0 if two else S["units"] & 1
                S["units"] += 1
                S.update(j=first_tile(S["count"]), end=nt, base=S["count"], count=S["count"] + nt)
                yield wait(q_full[S["q"]], S["units"] - 1 if two else S["units"] - 1 >> 1)
                if S["j"] >= S["end"]:
                    ops.append(("commit", q_empty[S["q"]]))
            if S["more"]:
                s, ph = k_at(S["base"] + S["j"])
                yield wait(kv_full[s], ph)

        def issue():
            t = S["base"] + S["j"]
            s, b = k_at(t)[0], S["items"] % nb
            ops.append(("S", t, s, S["q"], S["at"], b))
            ops.append(("commit", s_full[st][b]))
            ops.append(("commit", kv_empty[s]))
            S["items"] += 1
            S["j"] += step
            if S["j"] >= S["end"]:
                ops.append(("commit", q_empty[S["q"]]))

        for _ in range(ahead):
            yield from prepare()
            if S["more"]:
                issue()
        while True:
            while more_o and j_o >= end_o:
                if at_o >= 0:
                    release(at_o)
                at_o += 1
                yield from fetch(at_o)
                more_o = at_o < END
                nt = pieces[at_o] if more_o else 0
                if not more_o or nt == 0:
                    continue
                j_o, end_o, base_o, count_o, start = first_tile(count_o), nt, count_o, count_o + nt, True
            if not more_o:
                return
            t = base_o + j_o
            s, ph = v_at(t)
            yield wait(kv_full[s], ph)
            if start and sums >= nb:
                yield wait(o_empty[st][sums % nb], sums // nb - 1)
            yield from prepare()
            b = items_o % nb
            yield wait(p_full[st][b], items_o // nb)
            ops.append(("PV", t, s, at_o, b, sums % nb))
            ops.append(("commit", kv_empty[s]))
            start, j_o, items_o = False, j_o + step, items_o + 1
            if j_o >= end_o:
                ops.append(("commit", o_full[st][sums % nb]))
                sums += 1
            if S["more"]:
                issue()

    def softmax(st):
        items = tiles = n = 0
        sums, done = [0, 0], None

        def finish(d):
            at, k, counts, begun = d
            if counts is not None:
                if not two:
                    yield wait(meet, k)
                mine = [st] if two else [x for x in (0, 1) if counts[x]]
                for x in mine:
                    yield wait(o_full[x][begun[x] % nb], begun[x] // nb)
                for x in mine:
                    assert obuf[x][begun[x] % nb] == at, "O of another unit"
                yield lambda: True
                for x in mine:
                    assert obuf[x][begun[x] % nb] == at, "O of another unit"
                    o_empty[x][begun[x] % nb].arrive()
            release(at)

        at = 0
        while True:
            yield from fetch(at)
            assert ring[at % RING] == at
            if at == END:
                if done:
                    yield from finish(done)
                return
            nt = pieces[at]
            n0 = nt if two else (nt + 1 - (tiles & 1)) >> 1
            counts = [n0, nt if two else nt - n0]
            j = 0 if two else (tiles & 1) ^ st
            while j < nt:
                b = items % nb
                yield wait(s_full[st][b], items // nb)
                assert sbuf[st][b] == ("S", first[at] + j), "S of another tile"
                yield lambda: True
                sbuf[st][b] = ("P", first[at] + j)
                p_full[st][b].arrive()
                items, j = items + 1, j + (1 if two else 2)
                if layout.deferred and done:
                    yield from finish(done)
                    done = None
            tiles += nt
            if done:
                yield from finish(done)
            done = (at, n, counts if nt else None, list(sums))
            if nt:
                if not two:
                    meet.arrive()
                sums = [sums[0] + (counts[0] > 0), sums[1] + (counts[1] > 0)]
                n += 1
            if not layout.deferred:
                yield from finish(done)
                done = None
            at += 1

    def execute(st):
        op = pipe[st].pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "S":
            _, t, s, q, unit, b = op
            assert stage[s] == ("K", t), "K of another tile"
            assert qbuf[q] == unit, "Q of another unit"
            assert sbuf[st][b] is None or sbuf[st][b][0] == "done", "S over a P in use"
            sbuf[st][b] = ("S", t)
        else:
            _, t, s, unit, b, o = op
            assert stage[s] == ("V", t), "V of another tile"
            assert sbuf[st][b] == ("P", t), "P of another tile"
            sbuf[st][b] = ("done", t)
            obuf[st][o] = unit

    roles = {"scheduler": scheduler(), "producer": producer(), "issuer0": issuer(0), "issuer1": issuer(1),
             "softmax0": softmax(0), "softmax1": softmax(1)}
    blocked = dict.fromkeys(roles)
    while roles or copies or pipe[0] or pipe[1]:
        able = [("role", r) for r in roles if blocked[r] is None or blocked[r]()]
        able += [("copy", i) for i in range(len(copies))] + [("mma", st) for st in (0, 1) if pipe[st]]
        if not able:
            return "deadlock"
        kind, x = rng.choice(able)
        if kind == "role":
            try:
                blocked[x] = next(roles[x])
            except StopIteration:
                del roles[x]
        elif kind == "copy":
            what, to, data = copies.pop(x)
            if what == "q":
                qbuf[to] = data
                q_full[to].arrive()
            else:
                stage[to] = data
                kv_full[to].arrive()
        else:
            execute(x)
    return "ok"
