"""A model of the roles of the attention kernels over the 8-bit cache: who waits for whom.

Each role of a CTA (csrc/fa_kv8_fwd.cu: items of up to 16 rows; csrc/fa_kv8_rows.cu: items of 128)
is a generator that stops wherever it waits, the tensor core an engine that works in order, copies
land in any order, and a random schedule runs them.  Barriers are as the hardware's: a wait on an
mbarrier looks at the parity of its last complete phase only, a named barrier counts arrivals,
whoever they are from.  The warps of one role walk together here (their own barriers see to that).
`run` returns what went wrong first: a wait that passed for an older phase, keys or values used before
they landed or overwritten before they were read, a copy into a place with a copy in flight, a role
twice at a barrier, roles that wait for one another for good.  (With 128 rows there is a second warp
of the softmax, `tail`, that has no rows in some parts.)

`without` leaves out one of what the kernels do against these:
  empty parts     items whose rows see nothing are not handed out
  two products    the product barriers alternate by tile (narrow)
  first keys      the values' warps wait for a part's first keys too, before its queries (128 rows)
  queries' part   the queries' warp gives parts back, as the others do (narrow)
  issuer's waits  after an abort too, scores and products are waited for before a barrier's next turn
                  (128 rows)
  parts' ends     after an abort too, the softmax waits for a part's last product (128 rows)
  abort seen      the producer looks at the abort flag once a place is free
"""
from __future__ import annotations

import random

PARTS = 4     # parts handed out and not given back by all


class Wrong(Exception):
    pass


class Phases:
    """An mbarrier of `count` arrivals a phase."""

    def __init__(self, count):
        self.count = self.left = count
        self.done = 0          # complete phases

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.done += 1

    def passes(self, phase):
        return (self.done - 1) % 2 == phase % 2


class Meeting:
    """A named barrier."""

    def __init__(self, count):
        self.count, self.here, self.turn = count, [], 0

    def come(self, who):
        if who in self.here:
            raise Wrong("twice at a barrier")
        self.here.append(who)
        if len(self.here) == self.count:
            self.here, self.turn = [], self.turn + 1


class Cta:
    def __init__(self, kind, parts, slots, seed, without=(), abort_at=None):
        self.rng = random.Random(seed)
        self.without = {without} if isinstance(without, str) else set(without)
        self.narrow = kind == "narrow"
        self.parts = parts if "empty parts" in self.without else [p for p in parts if p]
        self.slots, self.abort_at, self.abort = slots, abort_at, False
        self.units = 1 if self.narrow else 2            # units of a tile's keys, and of its values
        self.without_rows = [self.rng.random() < 0.4 for _ in parts]   # of the softmax's second warp
        roles = 4                                       # that give parts back
        if "queries' part" in self.without and self.narrow:
            roles -= 1
        self.handed = [None] * PARTS
        self.part_full = [Phases(1) for _ in range(PARTS)]
        self.part_empty = [Phases(roles) for _ in range(PARTS)]
        self.full = [Phases(1) for _ in range(slots)]
        self.empty = [Phases(1) for _ in range(slots)]
        self.q_full = [Phases(1 if self.narrow else 3) for _ in range(2)]
        self.q_empty = [Phases(2 if self.narrow else 3) for _ in range(2)]
        self.s_full = [Phases(1), Phases(1)]
        self.product = [Phases(1), Phases(1)]           # of a tile (narrow) or of a half
        self.meetings, self.flight, self.queue = {}, [], []
        self.holds = [None] * slots                     # the unit that a place holds
        self.products_done = 0

    # ------------------------------------------------------------------ what roles do

    def wait(self, bar, phase):
        """Whether the phase completed (not after an abort)."""
        while not bar.passes(phase):
            if self.abort:
                return False
            yield
        if bar.done <= phase and not self.abort:
            raise Wrong("a wait passed for an older phase")
        return True

    def drain(self, bar, phase):
        while not bar.passes(phase):
            yield

    def meet(self, name, count, who):
        bar = self.meetings.setdefault(name, Meeting(count))
        turn = bar.turn
        bar.come(who)
        while bar.turn == turn:
            yield

    def come_to_half(self, half, ok, who, idle=False):
        if not idle and (ok or "issuer's waits" not in self.without):
            self.meetings.setdefault(half, Meeting(4)).come(who)
        else:
            yield from self.meet(half, 4, who)

    def wait_for_issuer(self, bar, phase, ok):
        if "issuer's waits" in self.without:
            return ok and (yield from self.wait(bar, phase))
        yield from self.drain(bar, phase)
        if bar.done != phase + 1:
            raise Wrong("a wait passed for another phase")
        return ok

    def take(self, np):
        yield from self.drain(self.part_full[np % PARTS], np // PARTS)
        if self.handed[np % PARTS][0] != np:
            raise Wrong("a part that is not the next")
        return self.handed[np % PARTS][1]

    def give(self, np):
        self.part_empty[np % PARTS].arrive()

    def unit(self, n):
        return self.full[n % self.slots], n // self.slots

    def use(self, n):
        if self.holds[n % self.slots] != n and not self.abort:
            raise Wrong("keys or values that are not there")

    # ------------------------------------------------------------------ both kernels

    def producer(self):
        n, ok = 0, True
        for np, tiles in enumerate(self.parts + [-1]):
            if np >= PARTS:
                yield from self.drain(self.part_empty[np % PARTS], np // PARTS - 1)
            self.handed[np % PARTS] = np, tiles
            self.part_full[np % PARTS].arrive()
            for _ in range(max(tiles, 0) * 2 * self.units):
                if ok and n >= self.slots:
                    ok = yield from self.wait(self.empty[n % self.slots], n // self.slots - 1)
                if ok and self.abort and "abort seen" not in self.without:
                    ok = False
                if not ok:
                    break
                if any(x % self.slots == n % self.slots for x in self.flight):
                    raise Wrong("a copy into a place with a copy in flight")
                self.flight.append(n)
                n += 1
                yield
        while self.flight:
            yield

    def land(self):
        n = self.flight.pop(self.rng.randrange(len(self.flight)))
        self.holds[n % self.slots] = n
        self.full[n % self.slots].arrive()

    def engine(self):
        what, x = self.queue.pop(0)
        if what == "commit":
            x.arrive()
        elif what == "product":
            self.products_done = x + 1
        else:
            self.use(x)

    def commit(self, bar):
        self.queue.append(("commit", bar))

    # ------------------------------------------------------------------ up to 16 rows

    def product_of(self, tile):
        return (self.product[0], tile) if "two products" in self.without else (self.product[tile % 2], tile // 2)

    def narrow_issuer(self):
        np, left, T = -1, 0, -1

        def advance():
            nonlocal np, left
            while left == 0:
                tiles = yield from self.take(np + 1)
                if tiles < 0:
                    return False
                np, left = np + 1, tiles
                self.give(np)
                if tiles == 0:
                    yield from self.wait(self.q_full[np % 2], np // 2)
                    self.commit(self.q_empty[np % 2])
            left -= 1
            return True

        more = yield from advance()
        if more:
            yield from self.meet("keys", 2, "issuer")
        while more or T >= 0:
            if more:
                self.queue.append(("use", 2 * T + 2))
                self.commit(self.s_full[(T + 1) % 2])
                self.commit(self.empty[(2 * T + 2) % self.slots])
                if left == 0:
                    self.commit(self.q_empty[np % 2])
            if T >= 0:
                yield from self.meet("weights", 2, "issuer")
                self.queue += [("use", 2 * T + 1), ("product", T)]
                self.commit(self.product_of(T)[0])
                self.commit(self.empty[(2 * T + 1) % self.slots])
                if not more:
                    break
            more = yield from advance()
            yield from self.meet("keys", 2, "issuer")
            T += 1

    def narrow_queries(self):
        np, ok = 0, True
        while (yield from self.take(np)) >= 0:
            if "queries' part" not in self.without:
                self.give(np)
            if np >= 2 and ok:
                ok = yield from self.wait(self.q_empty[np % 2], np // 2 - 1)
            if ok:
                self.q_full[np % 2].arrive()
            np += 1
            yield

    def narrow_relay(self):
        np = T = 0
        while (tiles := (yield from self.take(np))) >= 0:
            self.give(np)
            for i in range(tiles):
                if T > 0:
                    yield from self.wait(*self.unit(2 * T - 1))
                yield from self.wait(*self.unit(2 * T))
                if i == 0:
                    yield from self.wait(self.q_full[np % 2], np // 2)
                yield from self.meet("keys", 2, "relay")
                T += 1
            np += 1
        if T > 0:
            yield from self.wait(*self.unit(2 * T - 1))
            yield from self.meet("keys", 2, "relay")

    def narrow_softmax(self):
        np, T, ok = 0, 0, True
        while (tiles := (yield from self.take(np))) >= 0:
            if ok:
                ok = yield from self.wait(self.q_full[np % 2], np // 2)
            for _ in range(tiles):
                if ok:
                    ok = yield from self.wait(self.s_full[T % 2], T // 2)
                yield from self.meet("weights", 2, "softmax")
                T += 1
            if ok and tiles:
                ok = yield from self.wait(*self.product_of(T - 1))
                if ok and self.products_done < T and not self.abort:
                    raise Wrong("a product that is not complete")
            self.q_empty[np % 2].arrive()
            self.give(np)
            np += 1
            yield

    # ------------------------------------------------------------------ 128 rows

    def rows_issuer(self):
        np, with_tiles, left, T, first = -1, -1, 0, -1, True

        def advance():
            nonlocal np, with_tiles, left, first
            while left == 0:
                tiles = yield from self.take(np + 1)
                if tiles < 0:
                    return False
                np, left, first = np + 1, tiles, True
                with_tiles += tiles > 0
                self.give(np)
            left -= 1
            return True

        more = yield from advance()
        while more or T >= 0:
            if T >= 0:
                for half in range(2):
                    yield from self.meet(half, 4, "issuer")
                    self.queue.append(("product", 2 * T + half))
                    self.commit(self.product[half])
                if not more:
                    break
            if first:
                yield from self.wait(self.q_full[0], with_tiles)
                if "first keys" in self.without:
                    for u in range(2):
                        yield from self.wait(*self.unit(4 * T + 4 + u))
            for u in range(2):
                self.queue.append(("use", 4 * T + 4 + u))
            self.commit(self.s_full[0])
            for u in range(2):
                self.commit(self.empty[(4 * T + 4 + u) % self.slots])
            if left == 0:
                self.commit(self.q_empty[0])
            first = False
            more = yield from advance()
            T += 1

    def rows_values(self):
        np, cut, T, ok = 0, 0, 0, True
        while (tiles := (yield from self.take(np))) >= 0:
            self.give(np)
            np += 1
            if tiles == 0:
                continue
            if cut and ok:
                ok = yield from self.wait(self.q_empty[0], cut - 1)
            if "first keys" not in self.without:
                for n in (4 * T, 4 * T + 1):
                    if ok:
                        ok = yield from self.wait(*self.unit(n))
            self.q_full[0].arrive()
            cut += 1
            for i in range(tiles):
                for half in range(2):
                    n = 4 * T + 2 + half
                    if ok:
                        ok = yield from self.wait(*self.unit(n))
                    if T > 0:
                        ok = yield from self.wait_for_issuer(self.product[half], T - 1, ok)
                    if ok:
                        self.use(n)
                    self.empty[n % self.slots].arrive()
                    if half == 1 and i + 1 < tiles:
                        for m in (4 * T + 4, 4 * T + 5):
                            if ok:
                                ok = yield from self.wait(*self.unit(m))
                    yield from self.come_to_half(half, ok, "values")
                T += 1

    def rows_tail(self):
        yield from self.rows_softmax("tail")

    def rows_softmax(self, who="softmax"):
        np, cut, T, ok = 0, 0, 0, True
        while (tiles := (yield from self.take(np))) >= 0:
            if tiles:
                if cut and ok:
                    ok = yield from self.wait(self.q_empty[0], cut - 1)
                self.q_full[0].arrive()
                if ok:
                    ok = yield from self.wait(self.q_full[0], cut)
                self.q_empty[0].arrive()
                cut += 1
            idle = who == "tail" and self.without_rows[np]
            for _ in range(tiles):
                for half in range(2):
                    if half == 0 and not idle:
                        ok = yield from self.wait_for_issuer(self.s_full[0], T, ok)
                    yield from self.come_to_half(half, ok, who, idle)
                    yield
                T += 1
            if tiles and (ok or "parts' ends" not in self.without):
                if "parts' ends" in self.without:
                    ok = yield from self.wait(self.product[1], T - 1)
                else:
                    ok = yield from self.wait_for_issuer(self.product[1], T - 1, ok)
                if ok and self.products_done < 2 * T and not self.abort:
                    raise Wrong("a product that is not complete")
            self.give(np)
            np += 1
            yield

    # ------------------------------------------------------------------ the schedule

    def run(self, most=60000):
        names = ["queries", "relay", "softmax", "issuer"] if self.narrow else ["values", "softmax", "tail", "issuer"]
        prefix = "narrow_" if self.narrow else "rows_"
        roles = {"producer": self.producer(), **{n: getattr(self, prefix + n)() for n in names}}
        speed = {n: self.rng.choice([1, 3, 10]) for n in roles}
        speed |= dict(engine=self.rng.choice([1, 3, 10, 30]), land=self.rng.choice([0.3, 1, 3, 10]))
        try:
            for step in range(most):
                if not roles:
                    return "fine"
                if self.abort_at is not None and step >= self.abort_at:
                    self.abort = True
                free = [*roles, *(["engine"] if self.queue else []), *(["land"] if self.flight else [])]
                pick = self.rng.choices(free, [speed[n] for n in free])[0]
                if pick in roles:
                    try:
                        next(roles[pick])
                    except StopIteration:
                        del roles[pick]
                else:
                    getattr(self, pick)()
        except Wrong as e:
            return str(e)
        return "stuck"


def outcomes(kind, runs, without=(), abort=False, empty=False, slots=(4, 6, 8, 12)):
    """How often each outcome came up."""
    found = {}
    for seed in range(runs):
        rng = random.Random(seed)
        sizes = [1, 1, 1, 2, 3, 5] + ([0, 0, 0] if empty else [])
        parts = [rng.choice(sizes) for _ in range(rng.randint(1, 16))]
        at = int(2 ** rng.uniform(3, 12)) if abort else None
        x = Cta(kind, parts, rng.choice(slots), seed, without, at).run()
        found[x] = found.get(x, 0) + 1
    return found
