"""The barriers of the tensor-core kernel of attention over pages, as a model run under random schedules on the CPU.

A wait on an mbarrier names only a phase's parity.  It is sound when the barrier can neither be two phases ahead of
the one that the waiter means (it would block for a phase that may never come) nor two behind (it would pass early).
The model runs every warp of a CTA through the waits and arrivals of the kernel, with copies and products that end
at any later time, and checks that at every moment of every wait; a schedule that ends with a warp waiting is a
deadlock.  Slow warps are what a schedule varies most: a warp may lag as far as the barriers let it."""
import random

import pytest

MISTAKES = ("lapped accumulator", "lapped query tile")


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1


class Cta:
    """One CTA over `pieces`, each (cols, two, nt); NS ring slots; TP: no item of the other layout comes first."""

    def __init__(self, pieces, slots, rng, mistake=None):
        self.pieces, self.NS, self.rng, self.mistake = pieces, slots, rng, mistake
        self.TP = all(p[0] for p in pieces)
        b = self.b = {}
        for i in range(slots):
            b["full", i], b["empty", i] = Bar(1), Bar(2)
        for i in range(2):
            b["q_full", i], b["q_empty", i], b["o_free", i], b["fix", i], b["v_ready", i] = Bar(1), Bar(2), Bar(4), Bar(4), Bar(1)
            for j in range(2):
                b["s_full", i, j], b["p_full", i, j], b["pv_done", i, j] = Bar(1), Bar(4), Bar(1)
        for i in range(4):
            b["pc_full", i], b["pc_empty", i] = Bar(1), Bar(11)
        b["fix", 2], b["x_full",], b["x_free",] = Bar(8), Bar(4), Bar(4)
        self.copies = []           # copies in flight: barriers to arrive at, in any order
        self.products = ([], [])   # commits of each issuing warp, in order
        chance = rng.choice([0.0, 0.2, 0.8])
        # what the data decide, the same for every warp that they concern
        self.inner = lambda *k, m={}: m.setdefault(k, rng.random() >= chance)
        self.bad = lambda *k, m={}: m.setdefault(k, rng.random() < 0.3)
        self.move = lambda *k, m={}: m.setdefault(k, rng.random() < 0.2)
        self.joins = lambda *k, m={}: m.setdefault(k, rng.random() < 0.3)

    def arrive(self, *name):
        self.b[name].arrive()

    # every role yields the waits ((barrier name), phase)
    def loader(self):
        tiles = 0
        for seg in range(len(self.pieces) + 1):
            yield ("pc_full", seg & 3), seg >> 2
            if seg == len(self.pieces):
                return
            cols, two, nt = self.pieces[seg]
            ahead = 2 if cols else 0
            for u in range(nt + ahead):
                for kv in range(2):
                    if (u >= nt) if kv == 0 else (u < ahead):
                        continue
                    s = tiles % self.NS
                    if tiles >= self.NS:
                        yield ("empty", s), tiles // self.NS - 1
                    self.copies.append(("full", s))
                    tiles += 1
            self.arrive("pc_empty", seg & 3)

    def issue(self, g):
        commit = self.products[g].append
        tiles = job = qt = on = 0
        qn = [0, 0]
        NS = self.NS
        for seg in range(len(self.pieces) + 1):
            yield ("pc_full", seg & 3), seg >> 2
            if seg == len(self.pieces):
                return
            cols, two, nt = self.pieces[seg]
            self.arrive("pc_empty", seg & 3)
            ahead = 2 if cols else 0
            buf = g if two else qt
            for i in range(2):
                if two or qt == i:
                    yield ("q_full", i), qn[i]
            if two and self.mistake != "lapped query tile":
                self.arrive("q_empty", g ^ 1)  # this warp has seen the other's tile
            if self.mistake == "lapped accumulator":
                on = seg
            if not two and g >= nt:  # no tile for this group
                if self.mistake == "lapped accumulator" and on > 0:
                    yield ("o_free", g), on - 1
                self.arrive("q_empty", buf)
            if cols:
                kjob = job
                for u in range(nt + ahead):
                    if u < nt:
                        x = 2 * tiles + u + max(0, u - ahead)
                        yield ("full", x % NS), x // NS
                        if (u & 1) != g:
                            self.arrive("empty", x % NS)
                        else:
                            if not self.TP and kjob == job and kjob > 0:
                                yield ("pv_done", g, kjob - 1 & 1), kjob - 1 >> 1
                            commit(("s_full", g, kjob & 1))
                            commit(("empty", x % NS))
                            if self.TP and u + 2 >= nt:
                                commit(("q_empty", buf))
                            kjob += 1
                    if u >= ahead:
                        t = u - ahead
                        x = 2 * tiles + min(nt, t + ahead + 1) + t
                        yield ("full", x % NS), x // NS
                        if (t & 1) != g:
                            self.arrive("empty", x % NS)
                        else:
                            self.arrive("v_ready", g)
                            yield ("p_full", g, job & 1), job >> 1
                            if t == g and on > 0:
                                yield ("o_free", g), on - 1
                            commit(("pv_done", g, job & 1))
                            commit(("empty", x % NS))
                            if not self.TP and t + 2 >= nt:
                                commit(("q_empty", buf))
                            job += 1
            else:
                vp = -1
                for u in range(nt):
                    xk = 2 * (tiles + u)
                    sk, sv = xk % NS, (xk + 1) % NS
                    yield ("full", sk), xk // NS
                    if not two and (u & 1) != g:
                        self.arrive("empty", sk)
                        yield ("full", sv), (xk + 1) // NS
                        self.arrive("empty", sv)
                        continue
                    if job > 1:
                        yield ("pv_done", g, job - 2 & 1), job - 2 >> 1
                    commit(("s_full", g, 0))
                    if vp >= 0:
                        yield ("p_full", g, 1), job - 1 >> 1
                        commit(("pv_done", g, 1))
                        commit(("empty", vp))
                    if job > 0:
                        yield ("pv_done", g, job - 1 & 1), job - 1 >> 1
                    commit(("s_full", g, 1))
                    commit(("empty", sk))
                    if u + (1 if two else 2) >= nt:
                        commit(("q_empty", buf))
                        if two and self.mistake == "lapped query tile":
                            commit(("q_empty", buf))
                    yield ("full", sv), (xk + 1) // NS
                    self.arrive("v_ready", g)
                    yield ("p_full", g, 0), job >> 1
                    if u == (0 if two else g) and on > 0:
                        yield ("o_free", g), on - 1
                    commit(("pv_done", g, 0))
                    vp = sv
                    job += 2
                if vp >= 0:
                    yield ("p_full", g, 1), job - 1 >> 1
                    commit(("pv_done", g, 1))
                    commit(("empty", vp))
            on += two or g < nt
            tiles += nt
            for i in range(2):
                qn[i] += two or qt == i
            qt ^= not two

    def planner(self):
        qt, used = 0, [0, 0]
        for seg in range(len(self.pieces) + 1):
            if seg >= 4:
                yield ("pc_empty", seg & 3), (seg >> 2) - 1
            self.arrive("pc_full", seg & 3)
            if seg == len(self.pieces):
                return
            cols, two, nt = self.pieces[seg]
            for w in range(1 + two):
                buf = w if two else qt
                if used[buf] > 0:
                    yield ("q_empty", buf), used[buf] - 1
                yield None  # the copy takes its time
                self.arrive("q_full", buf)
                used[buf] += 1
            qt ^= not two

    def softmax(self, g, warp):
        job = vjob = xn = qt = on = 0
        ph = {("fix", g): 0, ("fix", 2): 0}
        sn, qn, handover = [0, 0], [0, 0], False

        def meet(name):
            self.arrive(*name)
            ph[name] += 1
            return name, ph[name] - 1

        for seg in range(len(self.pieces) + 1):
            yield ("pc_full", seg & 3), seg >> 2
            if seg == len(self.pieces):
                return
            cols, two, nt = self.pieces[seg]
            step, t0 = (1, 0) if two else (2, g)
            has = t0 < nt
            if self.mistake == "lapped accumulator":
                on = seg
            fx = ("fix", 2) if two else ("fix", g)
            if cols:
                yield meet(("fix", g))
            for t in range(t0, nt, step):
                for hf in range(1 if cols else 2):
                    first = t == t0 and hf == 0
                    sb = job & 1 if cols else hf
                    yield ("s_full", g, sb), sn[sb]
                    sn[sb] += 1
                    pv = None if first else (("pv_done", g, job - 1 & 1), job - 1 >> 1)
                    inner = self.inner(seg, t)
                    bad = not inner and self.bad(seg, t, hf)
                    free = (("o_free", g), on - 1) if first and on > 0 else None
                    if cols:
                        if handover:
                            for i in range(2):
                                if qn[i]:
                                    yield ("q_empty", i), qn[i] - 1
                            handover = False
                        move = first
                        if not first:
                            yield meet(("fix", g))
                            move = self.move(seg, t)
                        if move:
                            if pv:
                                yield pv
                            for _ in range(2 if first else 3):
                                yield meet(("fix", g))
                        if not inner:
                            if pv:
                                yield pv
                            yield ("v_ready", g), vjob
                            yield meet(("fix", g))
                            if bad:
                                if free:
                                    yield free
                                for _ in range(2):
                                    yield meet(("fix", g))
                        if pv:
                            yield pv
                    else:
                        live = self.move(seg, "rows", g, warp) or warp == 0
                        if live and self.move(seg, t, hf, g, warp) and pv:
                            yield pv
                        if not inner:
                            yield ("v_ready", g), vjob
                            yield meet(fx)
                            if bad:
                                if live:
                                    if pv:
                                        yield pv
                                    if free:
                                        yield free
                                yield meet(fx)
                    self.arrive("p_full", g, job & 1)
                    job += 1
                vjob += 1
            if has:
                yield ("pv_done", g, job - 1 & 1), job - 1 >> 1
                if cols:
                    yield meet(("fix", g))
            if not two:
                if g == 1:
                    if xn > 0:
                        yield ("x_free",), xn - 1
                    self.arrive("x_full")
                else:
                    yield ("x_full",), xn
                    self.arrive("x_free")
                xn += 1
            if two or g == 0:
                if cols:
                    yield meet(("fix", g))
                yield None  # the result is written
                self.arrive("o_free", g)
                if not two and (nt > 1 or self.mistake == "lapped accumulator"):
                    self.arrive("o_free", 1)
                if cols and self.joins(seg):
                    yield meet(("fix", g))
                    yield meet(("fix", g))
            handover = handover or not cols
            on += has
            for i in range(2):
                qn[i] += two or qt == i
            qt ^= not two
            self.arrive("pc_empty", seg & 3)

    def run(self):
        """None, or what went wrong."""
        rng = self.rng
        roles = {"loader": self.loader(), "planner": self.planner(), "issue 0": self.issue(0), "issue 1": self.issue(1)}
        roles.update({f"softmax {g}.{w}": self.softmax(g, w) for g in range(2) for w in range(4)})
        speed = {name: rng.choice([1.0, 1.0, 1.0, 0.02]) for name in roles}
        lag = rng.choice([0.02, 0.3, 1.0])  # of copies and products
        at = {name: None for name in roles}
        for name in roles:
            at[name] = next(roles[name], StopIteration)
        while True:
            ready, wrong = [], None
            for name, w in at.items():
                if w is StopIteration:
                    continue
                if w is None:
                    ready.append(name)
                    continue
                bar, phase = self.b[w[0]], w[1]
                passes = (bar.done - 1 & 1) == (phase & 1)
                if passes != (bar.done > phase):
                    return f"{name} waits for phase {phase} of {w[0]} at {bar.done} complete"
                if passes:
                    ready.append(name)
            async_ = [("copy", i) for i in range(len(self.copies))] + [("product", g) for g in range(2) if self.products[g]]
            if not ready and not async_:
                left = [n for n, w in at.items() if w is not StopIteration]
                return f"deadlock: {[(n, at[n]) for n in left]}" if left else wrong
            weights = [speed[n] for n in ready] + [lag] * len(async_)
            pick = rng.choices(ready + async_, weights)[0]
            if pick in at:
                at[pick] = next(roles[pick], StopIteration)
            elif pick[0] == "copy":
                self.b[self.copies.pop(pick[1])].arrive()
            else:
                self.b[self.products[pick[1]].pop(0)].arrive()


def pieces_of(rng):
    """Prefix items in the rows-as-rows layout, then suffix items in either one."""
    kind = rng.choice(["rows", "columns", "both"])
    rows = [(False, rng.random() < 0.5, rng.choice([1, 1, 1, 2, 3, 6])) for _ in range(rng.randint(1, 7))]
    cols = [(True, False, rng.choice([1, 1, 1, 2, 3, 7])) for _ in range(rng.randint(1, 7))]
    return rows if kind == "rows" else cols if kind == "columns" else rows + cols


def schedules(seed, count, mistake=None):
    rng = random.Random(seed)
    for _ in range(count):
        pieces = pieces_of(rng)
        wrong = Cta(pieces, rng.choice([5, 8]), rng, mistake).run()
        if wrong:
            return f"{pieces}: {wrong}"
    return None


@pytest.mark.parametrize("seed", range(8))
def test_no_wait_is_lapped_or_passes_early(seed):
    assert schedules(seed, 60) is None


@pytest.mark.parametrize("mistake", MISTAKES)
def test_the_model_sees(mistake):
    """Protocols with a fault: the issuing warp of a group without a tile waits for the accumulator of the piece
    before, which others may free once more meanwhile; a query tile that is refilled before both issuing warps
    have seen it."""
    assert any(schedules(seed, 60, mistake) for seed in range(20))
