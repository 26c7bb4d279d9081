"""Order of the hand-offs in the kernel for requests with many rows, on a model of its roles (CPU).

A block works through a list of runs: runs of two row tiles A and B, and runs of one (the warps of tile B
rotate the keys instead).  The model has every warp that waits or arrives as a process of its own, barriers
that count phases as mbarriers do (a wait sees the parity of a phase only), copies and matrix products
that finish late, and takes their steps in random order, some processes much slower than others.  Whatever a
step reads carries what it must be: a key tile, a half of the scores, a result with all its products.

Which arrivals a run of one row tile makes for tile B's result, and what its waits count, is read from the
kernel's source, so that the model follows the kernel; the orders it must rule out are those it finds when
told that such runs count for tile B too.
"""
import os
import random
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "position_independent_kv_critical_gb300", "csrc", "kernel_many_rows.cuh")


def rules_of_the_source():
    """{pv_arrives, group_frees: in a run of one row tile tile B's issuer of P V arrives on O_DONE, its warps on
    O_FREE; by_item: the waits on both count items, not the items the tile takes part in}"""
    with open(SOURCE) as f:
        text = f.read()
    branches = [m.group(1) for m in re.finditer(r"if \(w\.single && t == 1\) \{(.*?)continue;", text, re.S)]
    assert len(branches) == 2 and "take_item" not in branches[0] and "rotate_tiles" in branches[1], "the roles' loops moved"
    done = re.findall(r"MB_O_DONE \+ t\], (\w+) & 1", text)
    free = re.findall(r"MB_O_FREE \+ t\], \((\w+) - 1\) & 1", text)
    assert len(done) == 1 and len(free) == 1 and done == free, "the waits on tile B's result moved"
    if done[0] != "it":      # counted where the tile has taken part, not before
        assert len(re.findall(r"\+\+%s;" % done[0], text)) == 2 and not any(done[0] in b for b in branches)
    return dict(pv_arrives="MB_O_DONE" in branches[0], group_frees="MB_O_FREE" in branches[1], by_item=done[0] == "it")


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

    def arrive(self, n=1, tx=0):
        self.tx += tx
        for _ in range(n):
            self.pending -= 1
            self._turn()

    def landed(self):
        self.tx -= 1
        self._turn()

    def passed(self, parity):
        return (self.phase & 1) != parity & 1


class Block:
    """One block over `items`, a list of (single, key tiles)."""

    def __init__(self, items, masked, rules, rng):
        self.items, self.masked, self.rules, self.rng = items, masked, rules, rng
        two = lambda n: [Bar(n), Bar(n)]
        tiles = lambda n: [two(n), two(n)]
        self.item_full, self.item_empty = two(1), two(13)
        self.q_full, self.q_empty = Bar(1), Bar(2)
        self.k_full, self.k_raw, self.k_rot, self.k_empty = two(1), two(1), two(4), two(2)
        self.v_full, self.v_raw, self.v_empty = two(1), two(1), two(2)
        self.m_full, self.m_empty = two(1), two(8)
        self.s_full, self.p_full, self.pv_done = tiles(1), tiles(4), tiles(1)
        self.o_done, self.o_free = two(1), two(4)
        # what memory holds
        self.slot = [None, None]
        self.q = [None, None]
        self.k = [None, None]                      # (kind, tile); kind per rotating warp while one is turned
        self.v = [None, None]
        self.mask = [None, None]
        self.s = [[[None] * 4, [None] * 4], [[None] * 4, [None] * 4]]      # [tile][buffer][warp]
        self.o = ["free", "free"]                  # "free", or (item, P V done)
        self.took = [[True] * 4, [True] * 4]
        self.results = []
        self.copies = []                           # in flight, land in any order
        self.queues = {}                           # of each issuer: products and commits, in order

    # ---- processes: they yield a condition to wait for, or None
    def producer(self):
        kc, raw_end = 0, None
        for it, (single, n) in enumerate(self.items + [(None, 0)]):
            if it >= 2:
                yield lambda: self.item_empty[it & 1].passed((it >> 1) - 1)
            self.slot[it & 1] = (it, single, n)
            self.item_full[it & 1].arrive()
            if single is None:
                return
            if it > 0:
                yield lambda: self.q_empty.passed(it - 1)
            tiles = [0] if single else [0, 1]
            for t in tiles:
                self.q[t] = None
            self.q_full.arrive(tx=len(tiles))
            for t in tiles:
                self.copies.append((self.land_q, (t, it)))
            for _ in range(n):
                ks = kc & 1
                if kc >= 2:
                    yield lambda: self.k_empty[ks].passed((kc >> 1) - 1)
                bar = self.k_raw[ks] if single else self.k_full[ks]
                self.k[ks] = None
                bar.arrive(tx=1)
                self.copies.append((self.land_k, (ks, "raw" if single else "turned", kc, bar)))
                if self.masked:
                    if kc >= 2:
                        yield lambda: self.m_empty[ks].passed((kc >> 1) - 1)
                    self.mask[ks] = kc
                    self.m_full[ks].arrive()
                kc += 1
                yield None

    def land_q(self, t, it):
        self.q[t] = it
        self.q_full.landed()

    def land_k(self, ks, kind, kc, bar):
        self.k[ks] = [(kind, kc)] * 4
        bar.landed()

    def land_v(self, vs, kind, vc, bar):
        self.v[vs] = (kind, vc)
        bar.landed()

    def take(self, it):
        yield lambda: self.item_full[it & 1].passed(it >> 1)
        now = self.slot[it & 1]
        need(now[0] == it, "a role took another item")
        self.item_empty[it & 1].arrive()
        return now[1], now[2]

    def values(self):
        vc, raw_n = 0, [0, 0]
        for it in range(len(self.items) + 1):
            single, n = yield from self.take(it)
            if single is None:
                return
            for j in range(n):
                vs = vc & 1
                dirty = j == n - 1 and self.rng.random() < 0.7 or self.rng.random() < 0.2
                if vc >= 2:
                    yield lambda: self.v_empty[vs].passed((vc >> 1) - 1)
                bar = self.v_raw[vs] if dirty else self.v_full[vs]
                self.v[vs] = None
                bar.arrive(tx=1)
                self.copies.append((self.land_v, (vs, "raw" if dirty else "ready", vc, bar)))
                if dirty:
                    yield lambda: bar.passed(raw_n[vs])
                    raw_n[vs] += 1
                    need(self.v[vs] == ("raw", vc), "zeroed another value tile")
                    self.v[vs] = ("ready", vc)
                    self.v_full[vs].arrive()
                vc += 1
                yield None

    def issuer(self, qk, t):
        """Warps 8/11 (Q K^T) and 12/13 (P V): what they issue finishes later, in their order."""
        queue = self.queues[qk, t] = []
        hq = kc = own = 0
        raw_n, full_n = [0, 0], [0, 0]
        for it in range(len(self.items) + 1):
            single, n = yield from self.take(it)
            if single is None:
                return

            def wait_k(ks):
                counts, bar = (raw_n, self.k_rot[ks]) if single else (full_n, self.k_full[ks])
                at = counts[ks]
                counts[ks] += 1
                return lambda: bar.passed(at)

            if single and t == 1:
                for j in range(n):
                    ks = (kc + j) & 1
                    yield wait_k(ks) if qk else (lambda: self.v_full[ks].passed((kc + j) >> 1))
                    (self.k_empty if qk else self.v_empty)[ks].arrive()
                if qk:
                    yield lambda: self.q_full.passed(it)
                    self.q_empty.arrive()
                elif self.rules["pv_arrives"]:
                    self.o_done[1].arrive()
                kc += n
                continue
            if qk:
                yield lambda: self.q_full.passed(it)
            count = it if self.rules["by_item"] else own
            for q in range(2 * n):
                hg, kt, h = hq + q, kc + (q >> 1), q & 1
                ks, buf = kt & 1, hg & 1
                if qk:
                    if h == 0:
                        yield wait_k(ks)
                    if hg >= 2:
                        yield lambda: self.pv_done[t][buf].passed((hg - 2) >> 1)
                    queue.append((self.do_qk, (t, it, hg, kt)))
                    queue.append((self.s_full[t][buf].arrive, ()))
                    if h == 1:
                        queue.append((self.k_empty[ks].arrive, ()))
                else:
                    yield lambda: self.p_full[t][buf].passed(hg >> 1)
                    if h == 0:
                        yield lambda: self.v_full[ks].passed(kt >> 1)
                    if q == 0 and count > 0:
                        yield lambda: self.o_free[t].passed(count - 1)
                    queue.append((self.do_pv, (t, it, q, hg, kt)))
                    queue.append((self.pv_done[t][buf].arrive, ()))
                    if h == 1:
                        queue.append((self.v_empty[ks].arrive, ()))
                yield None
            queue.append((self.q_empty.arrive, ()) if qk else (self.o_done[t].arrive, ()))
            hq += 2 * n
            kc += n
            own += 1

    def do_qk(self, t, it, hg, kt):
        need(self.q[t] == it, "Q K^T read the queries of another run")
        need(self.k[kt & 1] == [("turned", kt)] * 4, "Q K^T read another key tile")
        need(all(x is None or x == ("spent", hg - 2) for x in self.s[t][hg & 1]), "Q K^T overwrote scores or weights")
        self.s[t][hg & 1] = [("S", hg)] * 4

    def do_pv(self, t, it, q, hg, kt):
        need(self.s[t][hg & 1] == [("P", hg)] * 4, "P V read other weights")
        need(self.v[kt & 1] == ("ready", kt), "P V read another value tile")
        if q == 0:
            need(self.o[t] == "free", "P V overwrote a result that was not read")
            self.took[t] = [False] * 4
        else:
            need(self.o[t] == (it, q), "P V added to another result")
        self.o[t] = (it, q + 1)
        self.s[t][hg & 1] = [("spent", hg)] * 4

    def softmax(self, t, w):
        hq = kc = own = 0
        raw_n = [0, 0]
        for it in range(len(self.items) + 1):
            single, n = yield from self.take(it)
            if single is None:
                return
            if single and t == 1:
                for _ in range(n):
                    ks = kc & 1
                    yield lambda: self.k_raw[ks].passed(raw_n[ks])
                    raw_n[ks] += 1
                    if self.masked:
                        yield lambda: self.m_full[ks].passed(kc >> 1)
                        need(self.mask[ks] == kc, "other exclusion bits")
                        self.m_empty[ks].arrive()
                    need(self.k[ks] is not None and self.k[ks][w] == ("raw", kc), "turned another key tile")
                    yield None
                    self.k[ks] = self.k[ks][:w] + [("turned", kc)] + self.k[ks][w + 1:]
                    self.k_rot[ks].arrive()
                    kc += 1
                if self.rules["group_frees"]:
                    self.o_free[1].arrive()
                continue
            count = it if self.rules["by_item"] else own
            for q in range(2 * n):
                hg, ks, buf = hq + q, (kc + (q >> 1)) & 1, (hq + q) & 1
                yield lambda: self.s_full[t][buf].passed(hg >> 1)
                if self.masked and q & 1 == 0:
                    yield lambda: self.m_full[ks].passed((kc + (q >> 1)) >> 1)
                    need(self.mask[ks] == kc + (q >> 1), "other exclusion bits")
                    self.m_empty[ks].arrive()
                need(self.s[t][buf][w] == ("S", hg), "softmax of other scores")
                yield None
                if q > 0 and self.rng.random() < 0.3:          # the result is rescaled
                    last = hg - 1
                    yield lambda: self.pv_done[t][last & 1].passed(last >> 1)
                    need(self.o[t] == (it, q), "rescaled a result with products under way")
                self.s[t][buf][w] = ("P", hg)
                self.p_full[t][buf].arrive()
                yield None
            yield lambda: self.o_done[t].passed(count)
            need(self.o[t] == (it, 2 * n), "a result was read before its last product")
            yield None
            need(self.o[t] == (it, 2 * n), "a result changed while it was read")
            self.took[t][w] = True
            if all(self.took[t]):
                self.o[t] = "free"
                self.results.append((it, t))
            self.o_free[t].arrive()
            hq += 2 * n
            kc += n
            own += 1

    def run(self):
        procs = [self.producer(), self.values()]
        procs += [self.issuer(qk, t) for qk in (True, False) for t in (0, 1)]
        procs += [self.softmax(t, w) for t in (0, 1) for w in range(4)]
        rng = self.rng
        speed = [10 ** rng.uniform(-2, 2) for _ in procs]
        waits = [lambda: True for _ in procs]
        landing, products = 10 ** rng.uniform(-2, 2), 10 ** rng.uniform(-2, 2)
        while procs:
            able = [i for i in range(len(procs)) if waits[i]()]
            queues = [q for q in self.queues.values() if q]
            weights = [speed[i] for i in able] + [landing] * len(self.copies) + [products] * len(queues)
            if not weights:
                raise Fault("stuck")
            pick = rng.choices(range(len(weights)), weights)[0]
            if pick < len(able):
                i = able[pick]
                try:
                    waits[i] = next(procs[i]) or (lambda: True)
                except StopIteration:
                    del procs[i], waits[i], speed[i]
            elif pick < len(able) + len(self.copies):
                what, args = self.copies.pop(pick - len(able))
                what(*args)
            else:
                what, args = queues[pick - len(able) - len(self.copies)].pop(0)
                what(*args)
        while any(self.queues.values()):
            what, args = next(q for q in self.queues.values() if q).pop(0)
            what(*args)
        expect = [(it, t) for it, (single, _) in enumerate(self.items) for t in ((0,) if single else (0, 1))]
        need(sorted(self.results) == expect, "results are missing")


def faults(items, rules, runs, seed, masked=None):
    found = {}
    for i in range(runs):
        rng = random.Random(seed * 100003 + i)
        try:
            Block(items, rng.random() < 0.5 if masked is None else masked, rules, rng).run()
        except Fault as e:
            found[str(e)] = found.get(str(e), 0) + 1
    return found


PAIR, SINGLE = False, True
LISTS = {
    "pairs": [(PAIR, 1), (PAIR, 2), (PAIR, 1), (PAIR, 1), (PAIR, 3)],
    "singles": [(SINGLE, 1), (SINGLE, 3), (SINGLE, 1), (SINGLE, 1), (SINGLE, 2)],
    "pair, single of one tile": [(PAIR, 1), (SINGLE, 1), (PAIR, 1)],
    "single, pair of one tile": [(SINGLE, 1), (PAIR, 1), (PAIR, 1)],
    "long pair, single of one tile, pair": [(PAIR, 4), (SINGLE, 1), (PAIR, 2)],
    "taking turns": [(SINGLE, 2), (PAIR, 1), (SINGLE, 1), (SINGLE, 1), (PAIR, 1), (PAIR, 2), (SINGLE, 1), (PAIR, 1)],
    "many singles before a pair": [(SINGLE, 1)] * 5 + [(PAIR, 1)] * 2 + [(SINGLE, 1)] * 2 + [(PAIR, 1)],
}


@pytest.mark.parametrize("name", LISTS)
def test_every_order_reads_what_it_must(name):
    assert not faults(LISTS[name], rules_of_the_source(), 150, seed=len(name))


def test_random_lists_of_runs():
    rules = rules_of_the_source()
    for seed in range(150):
        rng = random.Random(seed)
        items = [(rng.random() < 0.5, rng.choice([1, 1, 1, 2, 3, 5])) for _ in range(rng.randint(1, 9))]
        assert not faults(items, rules, 2, seed), items


def test_the_model_finds_the_orders_that_counting_every_item_leaves_open():
    open_rules = dict(pv_arrives=True, group_frees=True, by_item=True)
    found = faults(LISTS["pair, single of one tile"], open_rules, 300, seed=1)
    assert "a result was read before its last product" in found and "stuck" in found, found
    found = faults(LISTS["single, pair of one tile"], open_rules, 1500, seed=2)
    assert "a result was read before its last product" in found, found
    for name in ("pairs", "singles"):
        assert not faults(LISTS[name], open_rules, 100, seed=3)
