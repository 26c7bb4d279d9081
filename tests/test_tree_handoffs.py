"""Order of the hand-offs in the tree attention's kernel, on a model of its roles (CPU).

A block works through a list of runs: of two row tiles, where both chains take every unit, and of one, where they
take the units in turn.  The model has every warp that waits or arrives as a process of its own, barriers that count
phases as mbarriers do (a wait sees the parity of a phase only), copies that land in any order and matrix products
that finish late, and takes their steps in random order, some processes much slower than others.  Whatever a step
reads carries what it must be: a unit's keys, its scores, a result with all its products.

Stages, ring of hidden bits and arrivals are read from the kernel's source.  Told of fewer stages than a rotating
group's parity needs, of a shorter ring or of a missing arrival, the model finds what they keep apart.
"""
import os
import random
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "position_independent_kv_critical_gb300", "csrc", "kernel_tree.cuh")


def rules_of_the_source(d):
    with open(SOURCE) as f:
        text = f.read()
    m = re.search(r"NK = D == 128 \? (\d+) : (\d+), NV = D == 128 \? (\d+) : (\d+);", text)
    nk, nv = (int(m.group(1)), int(m.group(3))) if d == 128 else (int(m.group(2)), int(m.group(4)))
    assert re.search(r"kMeta = 2 \* NK;", text)
    counts = {n: int(c) for n, c in re.findall(r"mbar_init\(&bars\[SM::B_(\w+?)(?: \+ \w)?\], (\d+)\);", text)}
    assert counts["Q_EMPTY"] == counts["K_EMPTY"] == counts["V_EMPTY"] == counts["Q_FULL"] == 1, "the issuers moved"
    assert counts["P_FULL"] == counts["K_ROT"] == counts["V_FULL"] == counts["O_FREE"] == counts["ML"] == 4
    return dict(nk=nk, nv=nv, meta=2 * nk, free_both="arrive_warp(&bars[SM::B_O_FREE + 1])" in text)


class Fault(Exception):
    pass


def need(ok, what):
    if not ok:
        raise Fault(what)


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx, self.phase = 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, tx=0):
        need(self.pending > 0, "an arrival too many")
        self.tx += tx
        self.pending -= 1
        self._turn()

    def landed(self):
        self.tx -= 1
        self._turn()

    def passed(self, turn):
        """Whether a wait for the phase of number `turn` goes on: it sees the parity."""
        return (self.phase & 1) != (turn & 1)


class Block:
    """One block over `runs`, a list of (one row tile, units)."""

    def __init__(self, runs, rules, rng):
        self.runs, self.r, self.rng = runs, rules, rng
        nk, nv = rules["nk"], rules["nv"]
        many = lambda n, c: [Bar(c) for _ in range(n)]
        self.item_full, self.item_empty = many(2, 1), many(2, 18)
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.k_raw, self.k_rot, self.k_empty = many(nk, 1), many(nk, 4), many(nk, 1)
        self.v_raw, self.v_full, self.v_empty = many(nv, 1), many(nv, 4), many(nv, 1)
        self.s_full, self.p_full, self.pv_done = ([many(2, c) for _ in range(2)] for c in (1, 4, 1))
        self.o_done, self.o_free, self.ml = many(2, 1), many(2, 4), Bar(4)
        self.slot, self.q = [None, None], None
        self.k, self.v = [[None] * 4 for _ in range(nk)], [[None] * 4 for _ in range(nv)]
        self.meta = [None] * rules["meta"]
        self.s = [[[None] * 4 for _ in range(2)] for _ in range(2)]        # [chain][buffer][warp]
        self.o = [[None, 0, 4], [None, 0, 4]]                               # run, products, warps that have read it
        self.sums = [None] * 4
        self.results = {}
        self.copies, self.queues = [], [[], []]

    def units(self, single, n, kc, t):
        return n if not single else (n + (1 if kc & 1 == t else 0)) >> 1

    def take(self, it):
        yield lambda: self.item_full[it & 1].passed(it >> 1)
        need(self.slot[it & 1] and self.slot[it & 1][0] == it, "a run read before it is there")
        got = self.slot[it & 1]
        self.item_empty[it & 1].arrive()
        return got

    # ---- processes: they yield a condition to wait for, or None
    def producer(self, val):
        stages = self.r["nv"] if val else self.r["nk"]
        raw, empty, ring = (self.v_raw, self.v_empty, self.v) if val else (self.k_raw, self.k_empty, self.k)
        kc = 0
        for it, (single, n) in enumerate(self.runs + [(None, 0)]):
            if not val:
                if it >= 2:
                    yield lambda: self.item_empty[it & 1].passed((it >> 1) - 1)
                self.slot[it & 1] = (it, single, n)
                self.item_full[it & 1].arrive()
            for _ in range(n):
                st, turn = kc % stages, kc // stages
                if turn:
                    yield lambda: empty[st].passed(turn - 1)
                if not val:
                    self.meta[kc % self.r["meta"]] = kc
                ring[st] = [None] * 4
                raw[st].arrive(tx=1)
                self.copies.append((ring, st, kc, raw[st]))
                kc += 1
                yield None

    def rotation(self, group, warp):
        kc = it = 0
        while True:
            _, single, n = yield from self.take(it)
            if single is None:
                return
            for u in range(kc + (0 if kc & 1 == group else 1), kc + n, 2):
                ks, vs = u % self.r["nk"], u % self.r["nv"]
                yield lambda: self.k_raw[ks].passed(u // self.r["nk"])
                need(self.meta[u % self.r["meta"]] == u, "hidden bits of another unit")
                need(self.k[ks][warp] == ("raw", u), "keys rotated that are not there")
                self.k[ks][warp] = ("ready", u)
                yield None
                self.k_rot[ks].arrive()
                yield lambda: self.v_raw[vs].passed(u // self.r["nv"])
                need(self.v[vs][warp] == ("raw", u), "values cleaned that are not there")
                self.v[vs][warp] = ("ready", u)
                yield None
                self.v_full[vs].arrive()
            kc += n
            it += 1

    def scores(self):
        kc, it, hg = 0, 0, [0, 0]
        while True:
            _, single, n = yield from self.take(it)
            if single is None:
                return
            if it:
                yield lambda: self.q_empty.passed(it - 1)
            self.q = None
            self.q_full.arrive(tx=1)
            self.copies.append(("q", None, it, self.q_full))
            yield lambda: self.q_full.passed(it)
            need(self.q == it, "queries of another run")
            for u in range(kc, kc + n):
                ks = u % self.r["nk"]
                yield lambda: self.k_rot[ks].passed(u // self.r["nk"])
                chains = [u & 1] if single else [0, 1]
                for t in chains:
                    b = hg[t] & 1
                    if hg[t] >= 2:
                        yield lambda: self.pv_done[t][b].passed((hg[t] - 2) >> 1)
                    self.queues[0].append(("qk", t, b, ks, it, u))
                    self.queues[0].append(("commit", self.s_full[t][b]))
                    if t == chains[-1]:
                        self.queues[0].append(("commit", self.k_empty[ks]))
                    hg[t] += 1
                    yield None
            self.queues[0].append(("commit", self.q_empty))
            kc += n
            it += 1

    def products(self):
        kc, it, hg, own = 0, 0, [0, 0], [0, 0]
        while True:
            _, single, n = yield from self.take(it)
            if single is None:
                return
            begun = [False, False]
            for u in range(kc, kc + n):
                vs = u % self.r["nv"]
                yield lambda: self.v_full[vs].passed(u // self.r["nv"])
                chains = [u & 1] if single else [0, 1]
                for t in chains:
                    b = hg[t] & 1
                    yield lambda: self.p_full[t][b].passed(hg[t] >> 1)
                    if not begun[t] and own[t]:
                        yield lambda: self.o_free[t].passed(own[t] - 1)
                    self.queues[1].append(("pv", t, b, vs, it, u, begun[t]))
                    self.queues[1].append(("commit", self.pv_done[t][b]))
                    if t == chains[-1]:
                        self.queues[1].append(("commit", self.v_empty[vs]))
                    begun[t] = True
                    hg[t] += 1
                    yield None
            for t in range(2):
                if begun[t]:
                    self.queues[1].append(("commit", self.o_done[t]))
                    own[t] += 1
            kc += n
            it += 1

    def softmax(self, t, warp):
        kc = it = hg = own = joined = 0
        while True:
            _, single, n = yield from self.take(it)
            if single is None:
                return
            mine, other = self.units(single, n, kc, t), self.units(single, n, kc, 1 - t)
            u = kc + (1 if single and kc & 1 != t else 0)
            for q in range(mine):
                b = hg & 1
                yield lambda: self.s_full[t][b].passed(hg >> 1)
                need(self.meta[u % self.r["meta"]] == u, "hidden bits of another unit")
                need(self.s[t][b][warp] == ("s", it, u), "scores read that are not there")
                if q and self.rng.random() < 0.3:                 # the reference moves: O is rescaled
                    yield lambda: self.pv_done[t][1 - b].passed((hg - 1) >> 1)
                    need(self.o[t][:2] == [it, q], "a result rescaled before its products")
                self.s[t][b][warp] = ("p", it, u)
                yield None
                self.p_full[t][b].arrive()
                hg += 1
                u += 2 if single else 1
            if mine:
                yield lambda: self.o_done[t].passed(own)
                own += 1
            if single and t == 1:
                if mine:
                    self.sums[warp] = it
                    yield None
                    self.ml.arrive()
            else:
                two = single and other > 0
                if two:
                    yield lambda: self.ml.passed(joined)
                    joined += 1
                    need(self.sums[warp] == it, "sums of another run")
                for c, k in ((t, mine), (1, other if two else 0)):
                    if k:
                        need(self.o[c][:2] == [it, k], "a result read before its last product")
                        self.o[c][2] += 1
                yield None
                if mine:
                    self.o_free[t].arrive()
                if two and self.r["free_both"]:
                    self.o_free[1].arrive()
                self.results.setdefault(it, []).append((t, warp))
            kc += n
            it += 1

    # ---- what finishes late
    def land(self):
        ring, st, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
        if ring == "q":
            self.q = what
        else:
            ring[st] = [("raw", what)] * 4
        bar.landed()

    def execute(self, i):
        op = self.queues[i].pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "qk":
            _, t, b, ks, it, u = op
            need(self.k[ks] == [("ready", u)] * 4, "scores of keys that are not there")
            need(self.q == it, "scores of another run's queries")
            self.s[t][b] = [("s", it, u)] * 4
        else:
            _, t, b, vs, it, u, more = op
            need(self.s[t][b] == [("p", it, u)] * 4, "weights that are not there")
            need(self.v[vs] == [("ready", u)] * 4, "values that are not there")
            if not more:
                need(self.o[t][2] == 4, "a result overwritten before it was read")
                self.o[t] = [it, 0, 0]
            need(self.o[t][0] == it, "a product of another run")
            self.o[t][1] += 1

    def run(self):
        rng = self.rng
        procs = [self.producer(False), self.producer(True), self.scores(), self.products()]
        procs += [self.rotation(g, w) for g in range(2) for w in range(4)]
        procs += [self.softmax(t, w) for t in range(2) for w in range(4)]
        speed = [rng.choice((0.02, 0.3, 1.0)) for _ in procs]
        late = [rng.choice((0.02, 0.3, 1.0)) for _ in range(3)]
        waits = [None] * len(procs)
        idle = 0
        while any(p is not None for p in procs):
            moved = False
            for i in rng.sample(range(len(procs)), len(procs)):
                if procs[i] is None or rng.random() > speed[i]:
                    continue
                if waits[i] is not None and not waits[i]():
                    continue
                moved = True
                try:
                    waits[i] = next(procs[i])
                except StopIteration:
                    procs[i] = None
            if self.copies and rng.random() < late[0]:
                self.land()
                moved = True
            for i in range(2):
                if self.queues[i] and rng.random() < late[1 + i]:
                    self.execute(i)
                    moved = True
            idle = 0 if moved else idle + 1
            need(idle < 3000, "a wait that never ends")
        for it, (single, n) in enumerate(self.runs):
            want = 4 if single else 8
            need(len(self.results.get(it, [])) == want, "a result is missing")


def some_runs(rng):
    return [(rng.random() < 0.5, rng.choice((1, 1, 1, 2, 3, 5, 9))) for _ in range(rng.randint(1, 9))]


def faults(rules, seeds):
    found = set()
    for seed in seeds:
        rng = random.Random(seed)
        try:
            Block(some_runs(rng), rules, rng).run()
        except Fault as e:
            found.add(str(e))
    return found


@pytest.mark.parametrize("d", [64, 128])
def test_every_order_is_right(d):
    assert faults(rules_of_the_source(d), range(150)) == set()


def test_many_runs_of_one_unit():
    rules = rules_of_the_source(128)
    for seed in range(60):
        rng = random.Random(1000 + seed)
        runs = [(rng.random() < 0.7, 1) for _ in range(25)]
        Block(runs, rules, rng).run()


@pytest.mark.parametrize("change", [dict(nk=5), dict(nv=3), dict(meta=4), dict(free_both=False)])
def test_the_model_finds_what_the_rules_keep_apart(change):
    assert faults({**rules_of_the_source(128), **change}, range(80))
