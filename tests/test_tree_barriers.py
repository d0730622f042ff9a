"""The barriers of tree_decode's kernel, modelled on the CPU.

A wait on an mbarrier names a phase by its parity alone: it is right when the phase waited for is the one under way or
the one before.  The model runs the kernel's roles -- two softmax streams, two MMA issuers, four producers, and the
copies and products that complete by themselves -- over barriers that count phases, in random orders and with one role
starved at a time, and fails when a wait is further away from its barrier, when an arrival comes too many, when a
buffer is used before or after its time, when nobody can go on, or when a copy or product is under way at the end.  Once
a wait has given up, every wait but the last ones (for copies and products in flight) returns at once: issuers and
producers whose phase was not complete stop, the softmax streams go on, and what S, P and Q hold no longer
matters.  What the ring's slots hold always does.
"""

import random

import pytest

TILES = 229376   # bytes of shared memory for the Q tiles and the ring


class Shape:
    def __init__(self, qp, pp):
        self.split = qp == 3 and pp == 3
        self.tt = 64 if pp == 1 or self.split else 32
        slots = (TILES - (2 if qp == 1 else 3) * 32768) // (self.tt * 256)
        self.ks = (slots * 2 // 5 + 1) & ~1
        self.vs = slots - self.ks
        self.rows = 256 if qp == 1 else 128
        self.flush = 0 if pp == 1 else 256 // self.tt


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0          # the phase under way
        self.tx = 0             # copies of this phase that have not landed

    def arrive(self, tx=0):
        assert self.left > 0, "an arrival too many"
        self.left -= 1
        self.tx += tx
        self.turn()

    def landed(self):
        self.tx -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase, self.left = self.phase + 1, self.count

    def done(self, phase, strict=True):
        """What a wait for `phase` is told; its parity must not stand for another phase."""
        assert not strict or phase in (self.phase, self.phase - 1), f"waits for phase {phase} while {self.phase} is under way"
        return (self.phase - 1 - phase) % 2 == 0


class Meet:
    """bar.sync of the two softmax streams."""

    def __init__(self):
        self.n, self.turns = 0, 0

    def come(self):
        self.n += 1
        if self.n == 2:
            self.n, self.turns = 0, self.turns + 1


class Kernel:
    """segments: (tiles, both streams hold different lists, tiles at the end that are special)."""

    def __init__(self, shape, segments, rng, one_q_ready=False, one_fixed=False, give_up_at=None,
                 copies_go_on=False, segments_go_on=False):
        self.sh, self.segments, self.rng = shape, segments, rng
        self.one_q, self.one_fixed, self.copies_go_on = one_q_ready, one_fixed, copies_go_on
        self.segments_go_on = segments_go_on
        self.give_up_at, self.abort = give_up_at, False   # the number of moves after which a wait gives up
        b2 = lambda n: [[Bar(n), Bar(n)] for _ in range(2)]
        self.k_full, self.k_empty = [Bar(1) for _ in range(shape.ks)], [Bar(2) for _ in range(shape.ks)]
        self.v_full, self.v_empty = [Bar(1) for _ in range(shape.vs)], [Bar(2) for _ in range(shape.vs)]
        self.q_ready = [Bar(2), Bar(2)]
        self.s_full, self.p_ready, self.o_done = b2(1), b2(1), b2(1)
        self.s_free = [Bar(1), Bar(1)]
        self.fixed = b2(1)
        self.meet = Meet()
        self.k_tile, self.v_tile = [None] * shape.ks, [None] * shape.vs   # what a slot holds
        self.sp = [[None, None], [None, None]]     # what a stream's S and P buffers hold
        self.p = [None, None]                      # split: P on its own
        self.q = [None, None]                      # the segment whose lists Q holds for a stream
        self.pipe = [[], []]                       # MMAs and commits of an issuer, in order
        self.copies = []

    # ---- roles: generators that yield None for a step, (barrier, phase) for a wait, which is answered with whether the
    # phase was complete, or a condition for a wait that does not give up
    def softmax(self, s):
        sh, done, tiles_done = self.sh, 0, 0
        for seg, (ntile, dual, nspecial) in enumerate(self.segments):
            steps = ntile if dual else (ntile // 2 if s else (ntile + 1) // 2)
            yield from self.together()
            for t in ((s,) if dual else (0, 1)):
                self.q[t] = seg
            yield None
            self.q_ready[0].arrive()
            if not self.one_q and (dual or ntile > 1):
                self.q_ready[1].arrive()
            yield None
            for i in range(steps):
                at = i if dual else 2 * i + s
                step, num, special = done + i, tiles_done + at, at >= ntile - nspecial
                buf = 0 if sh.split else step & 1
                if sh.flush and i > 0 and i % sh.flush == 0:
                    yield from self.products_done(s, step - 1)
                phase = step if sh.split else step >> 1
                yield self.s_full[s][buf], phase
                self.holds(self.sp[s][buf] == ("S", step))
                if sh.split:
                    self.s_free[s].arrive()
                if i > 0 and self.rng.random() < 0.3:       # a maximum grew
                    yield from self.products_done(s, step - 1)
                if not sh.split:
                    self.sp[s][buf] = ("P", step)
                    yield None
                odd = False
                if special:
                    yield self.v_full[num % sh.vs], num // sh.vs
                    self.holds(self.v_tile[num % sh.vs] == num)   # a stream that goes on may come before its tile
                    if dual:
                        for _ in range(4):
                            yield from self.together()
                    odd = self.rng.random() < 0.3
                if not sh.split:
                    self.p_ready[s][buf].arrive()
                    yield None
                    if special and odd:
                        yield from self.products_done(s, step)
                        self.holds(self.sp[s][buf] == ("P", step))   # P is read once more
                    if special and i + 2 < steps:
                        self.arrive_fixed(s, step)
                else:
                    for c in range(2):
                        if c or step:
                            yield self.o_done[s][0], 2 * step + c - 1
                        self.p[s] = (step, c)
                        yield None
                        self.p_ready[s][0].arrive()
                        yield None
                        if special and odd:
                            yield self.o_done[s][0], 2 * step + c
                            self.holds(self.p[s] == (step, c))
            if steps:
                yield from self.products_done(s, done + steps - 1)
            done, tiles_done = done + steps, tiles_done + ntile
            if not dual:
                yield from self.together()

    def arrive_fixed(self, s, step):
        self.fixed[s][0 if self.one_fixed else step & 1].arrive()

    def products_done(self, s, step):
        if self.sh.split:
            yield self.o_done[s][0], 2 * step + 1
        else:
            yield self.o_done[s][step & 1], step >> 1

    def together(self):   # bar.sync does not give up: both streams come to every one of them
        turn = self.meet.turns
        self.meet.come()
        yield lambda: self.meet.turns > turn

    def holds(self, right):
        assert right or self.abort, "a buffer does not hold what its user expects"

    def issuer(self, s):
        yield from self.issue(s)     # until all is issued, or a wait gives up
        yield lambda: not self.pipe[s]

    def issue(self, s):
        sh, tiles_done, done, segs, fixes = self.sh, 0, 0, 0, [0, 0]
        for seg, (ntile, dual, nspecial) in enumerate(self.segments):
            stride, first = (1, 0) if dual else (2, s)
            steps = (ntile - first + stride - 1) // stride
            if self.one_q:
                if not (yield self.q_ready[0], seg):
                    return
            elif steps:
                if not (yield self.q_ready[s], segs) or (self.abort and not self.segments_go_on):
                    return
                segs += 1

            def scores(i):
                n, step = tiles_done + first + stride * i, done + i
                slot, buf = n % sh.ks, 0 if sh.split else step & 1
                if not (yield self.k_full[slot], n // sh.ks):
                    return False

                def mma():
                    assert self.k_tile[slot] == n
                    self.holds(self.q[s if dual else 0] == seg)
                    self.sp[s][buf] = ("S", step)
                self.pipe[s] += [mma, self.s_full[s][buf].arrive] + [self.k_empty[slot].arrive] * (1 if dual else 2)
                yield None
                return True

            def products(i, c=None):
                n, step = tiles_done + first + stride * i, done + i
                slot = n % sh.vs

                def mma():
                    assert self.v_tile[slot] == n
                    self.holds((self.p[s] == (step, c)) if sh.split else (self.sp[s][step & 1] == ("P", step)))
                self.pipe[s] += [mma, self.o_done[s][0 if sh.split else step & 1].arrive]
                if c != 0:
                    self.pipe[s] += [self.v_empty[slot].arrive] * (1 if dual else 2)
                yield None

            if not sh.split:
                for i in range(-2, steps):
                    at = first + stride * i
                    if i >= 0:
                        n, step = tiles_done + at, done + i
                        if not (yield self.v_full[n % sh.vs], n // sh.vs) or not (yield self.p_ready[s][step & 1], step >> 1):
                            return
                        yield from products(i)
                    if i + 2 < steps:
                        if i >= 0 and at >= ntile - nspecial and not (yield from self.wait_fixed(s, done + i, fixes)):
                            return
                        if not (yield from scores(i + 2)):
                            return
            else:
                for i in range(-1, steps):
                    if i + 1 < steps:
                        if done + i + 1 > 0 and not (yield self.s_free[s], done + i):
                            return
                        if not (yield from scores(i + 1)):
                            return
                    if i < 0:
                        continue
                    n, step = tiles_done + first + stride * i, done + i
                    if not (yield self.v_full[n % sh.vs], n // sh.vs):
                        return
                    for c in range(2):
                        if not (yield self.p_ready[s][0], 2 * step + c):
                            return
                        yield from products(i, c)
            tiles_done, done = tiles_done + ntile, done + steps

    def wait_fixed(self, s, step, fixes):
        buf = 0 if self.one_fixed else step & 1
        fixes[buf] += 1
        return (yield self.fixed[s][buf], fixes[buf] - 1)

    def producer(self, is_v, odd):
        full, empty, tile = (self.v_full, self.v_empty, self.v_tile) if is_v else (self.k_full, self.k_empty, self.k_tile)
        slots, n, stop = len(full), 0, False
        for n in range(sum(ntile for ntile, _, _ in self.segments)):
            if n % 2 != odd:
                continue
            slot, at = n % slots, n // slots
            if at > 0 and not (yield empty[slot], at - 1) and not self.copies_go_on:
                stop = True
                break
            full[slot].arrive(tx=1)
            self.copies.append((full[slot], tile, slot, n))
            yield None
        end = n if stop else n + 1
        for i in range(max(0, end - slots), end):
            if i % 2 == odd:
                if self.copies_go_on:
                    yield full[i % slots], i // slots
                else:
                    yield lambda: full[i % slots].done(i // slots)

    # ---- what completes by itself
    def hardware(self, which):
        if which < 2:
            if self.pipe[which]:
                self.pipe[which].pop(0)()
                return True
        elif self.copies:
            bar, tile, slot, n = self.copies.pop(self.rng.randrange(len(self.copies)))
            tile[slot] = n
            bar.landed()
            return True
        return False

    def run(self, starve=None):
        roles = {("softmax", s): self.softmax(s) for s in range(2)}
        roles.update({("issuer", s): self.issuer(s) for s in range(2)})
        roles.update({("producer", v, o): self.producer(v, o) for v in range(2) for o in range(2)})
        waits = {r: next(g, "end") for r, g in roles.items()}
        keys = list(roles) + [("hardware", 0), ("hardware", 1), ("hardware", 2)]

        def move(r):
            if r[0] == "hardware":
                return self.hardware(r[1])
            w, answer = waits[r], None
            if w == "end":
                return False
            if isinstance(w, tuple):
                answer = w[0].done(w[1], not self.abort)
                if not answer and not self.abort:
                    return False
            elif w is not None and not w():
                return False
            try:
                waits[r] = roles[r].send(answer)
            except StopIteration:
                waits[r] = "end"
            return True

        moves = 0
        while any(w != "end" for w in waits.values()):
            moves += 1
            self.abort = self.abort or moves == self.give_up_at
            order = [r for r in keys if r != starve]
            self.rng.shuffle(order)
            if not any(move(r) for r in order) and not (starve is not None and move(starve)):
                break
        assert all(w == "end" for w in waits.values()), {r: "waits" for r, w in waits.items() if w != "end"}
        assert not self.copies and not any(self.pipe), "under way at the end"


SHAPES = [(1, 1), (3, 1), (1, 3), (3, 3)]
STARVED = [None, ("softmax", 0), ("softmax", 1), ("issuer", 0), ("issuer", 1), ("producer", 0, 1), ("producer", 1, 0),
           ("hardware", 0), ("hardware", 1), ("hardware", 2)]


def draw_segments(rng, shape, special):
    out = []
    for _ in range(rng.randint(3, 14)):
        ntile = 1 if rng.random() < 0.4 else rng.randint(1, 20)
        out.append((ntile, shape.rows > 128 and rng.random() < 0.5, min(ntile, rng.choice(special))))
    return out


@pytest.mark.parametrize("starve", STARVED)
@pytest.mark.parametrize("qp,pp", SHAPES)
def test_waits_are_at_most_a_phase_away(qp, pp, starve):
    shape = Shape(qp, pp)
    assert shape.ks % 2 == 0 and shape.vs % 2 == 0
    for seed in range(4):
        rng = random.Random(seed)
        Kernel(shape, draw_segments(rng, shape, [0, 1, 2, 3, 9]), rng).run(starve)
    # runs of units of one tile, with longer ones behind them
    for seed in range(3):
        rng = random.Random(seed)
        Kernel(shape, [(1, False, 0)] * 30 + [(9, False, 0)] + [(1, False, 0)] * 7 + [(4, False, 0)] * 2, rng).run(starve)


def test_one_barrier_for_both_issuers_would_not_do():
    """The model sees the fault that q_ready's two barriers are there for."""
    rng = random.Random(0)
    with pytest.raises(AssertionError, match="waits for phase"):
        Kernel(Shape(1, 1), [(1, False, 0)] * 5 + [(6, False, 0)], rng, one_q_ready=True).run(("issuer", 1))


def test_one_barrier_for_both_buffers_would_not_do():
    """The same for `fixed`: two special steps in a row with more behind them."""
    rng = random.Random(0)
    with pytest.raises(AssertionError, match="waits for phase"):
        Kernel(Shape(1, 1), [(12, True, 9)] * 3, rng, one_fixed=True).run(("issuer", 0))


@pytest.mark.parametrize("starve", STARVED)
@pytest.mark.parametrize("qp,pp", SHAPES)
def test_a_wait_that_gives_up_leaves_nothing_under_way(qp, pp, starve):
    shape = Shape(qp, pp)
    for seed in range(12):
        rng = random.Random(seed)
        Kernel(shape, draw_segments(rng, shape, [0, 1, 3]), rng, give_up_at=rng.randint(1, 150)).run(starve)


def faults(starved, seeds, **kw):
    """What goes wrong over a number of runs."""
    seen = set()
    for seed in range(seeds):
        rng = random.Random(seed)
        shape = Shape(1, 1)
        try:
            Kernel(shape, draw_segments(rng, shape, [0, 1, 3]), rng, give_up_at=rng.randint(1, 100), **kw).run(starved)
        except AssertionError as e:
            seen.add(str(e).split("\n")[0])
    return seen


def test_copies_behind_a_wait_that_gave_up_would_not_do():
    """The model sees what producers that went on would do: a second arrival while a slot's copies are in flight."""
    assert "an arrival too many" in faults(("hardware", 2), 60, copies_go_on=True)


def test_segments_behind_a_wait_that_gave_up_would_not_do():
    """Softmax streams that go on announce the next segment's queries though the other stream's tiles are not there: an
    issuer that began it could take a slot's phase for the one after."""
    assert faults(("producer", 0, 1), 200, segments_go_on=True)
    assert not faults(("producer", 0, 1), 200)
