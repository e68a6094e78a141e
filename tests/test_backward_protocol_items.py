"""The tensor-core backward's barriers between the items of a CTA, and its way out
when a wait gives up: a model on the CPU beside test_backward_protocol's, with cells
for what outlives a tile. The roles run as coroutines in random order; copies and
tensor-core work end late but, per issuing warp, in order.

Beside the stages and score buffers it holds: the two kept operands (staged by a
warpgroup each, read by every score product of their item, or chunk), the
accumulators (begun by an item's first gradient product, read by both warpgroups), the
arrays in which rows_kernel's warpgroups join their partial sums, and dbias_kernel's
row vectors. Every wait of the kernels can be left out, which the model has to notice,
and every wait is bounded: where the copies stop coming, all roles have to end, with
no barrier overrun and no meeting left with one side. (What is read and written once a
wait has given up does not matter: the result is void.)"""
import random

import pytest

import test_backward_protocol
from test_backward_protocol import WARPGROUPS, Barrier, Queue


class Model:
    def __init__(self, kernel, items, nkt, seed, slots=True, stages=4, without=(), stall=None, arrays=2):
        self.rng = random.Random(seed)
        self.kernel, self.items, self.nkt, self.slots, self.stages = kernel, items, nkt, slots, stages
        self.without, self.stall, self.arrays = without, stall, arrays
        self.T = 2 * nkt if kernel == "rows" else nkt
        self.full, self.empty = [Barrier(1) for _ in range(stages)], [Barrier(1) for _ in range(stages)]
        self.s_full, self.r_full = [Barrier(1) for _ in range(2)], [Barrier(1) for _ in range(2)]
        self.p_full, self.g_done = [Barrier(1) for _ in range(8)], [Barrier(1) for _ in range(3)]
        self.a_ready, self.o_done = Barrier(WARPGROUPS), Barrier(1)
        self.live = True  # nothing has given up yet: what a cell holds matters
        model = self

        class Cell(test_backward_protocol.Cell):
            def write(self, tile, readers):
                if model.live:
                    super().write(tile, readers)

            def read(self, tile):
                if model.live:
                    super().read(tile)
        self.stage = [Cell(f"stage {s}") for s in range(stages)]
        self.buf, self.slot = [Cell(f"buffer {b}") for b in range(2)], [Cell(f"slot {s}") for s in range(3)]
        self.kept = [Cell(f"kept operand {w}") for w in range(WARPGROUPS)]
        self.vectors = [Cell(f"row vectors {w}") for w in range(WARPGROUPS)]
        self.acc = Cell("accumulators")
        self.acc_left = 0
        self.joins = {(a, w): Cell(f"join array {a} of {w}") for a in range(arrays) for w in range(WARPGROUPS)}
        self.copies, self.mma, self.mma2 = Queue(), Queue(), Queue()
        self.met = {"n": 0, "gen": 0}
        self.abort = False

    # ---- what the roles share
    def grads_of(self, t):
        return t >= self.nkt if self.kernel == "rows" else self.kernel == "cols"

    def where(self, g):
        T = self.T
        return (g // T * self.nkt + g % T - self.nkt) % 3 if self.slots and self.kernel == "rows" else g % 2

    def wait(self, name, barrier, k):
        """A bounded wait for the k-th completion; yields True or, given up, False."""
        if name in self.without:
            return True
        ok = yield ("wait", lambda: barrier.done(k))
        return ok

    def meet(self, name):
        if name in self.without:
            return
        gen = self.met["gen"]
        self.met["n"] += 1
        if self.met["n"] == WARPGROUPS:
            self.met["n"], self.met["gen"] = 0, gen + 1
        yield ("meet", lambda: self.met["gen"] > gen)

    # ---- roles
    def tma(self):
        g = 0
        for _ in range(self.items):
            for t in range(self.T):
                if self.stall is not None and g >= self.stall:
                    return  # the copies stop coming
                s = g % self.stages
                if g >= self.stages and not (yield from self.wait("empty", self.empty[s], g // self.stages - 1)):
                    return

                def land(s=s, g=g, n=2 + bool(self.grads_of(t))):
                    self.stage[s].write(g, n)
                    self.full[s].arrive()
                self.copies.put(land)
                g += 1

    def scores(self, it, g):
        b, s = g % 2, g % self.stages

        def run():
            self.stage[s].read(g)
            for k in self.kept:
                k.read(it)
            self.buf[b].write(g, 1)
        self.mma.put(run)
        self.mma.put(self.s_full[b].arrive)

    def grads(self, q, it, g, t, first):
        def run():
            self.stage[g % self.stages].read(g)
            self.slot[self.where(g)].read(g)
            if first:
                self.acc.write(it, WARPGROUPS)
                self.acc_left = self.T - (self.nkt if self.kernel == "rows" else 0)
            assert self.acc.tile == it or not self.live, "accumulators of another item"
            self.acc_left -= 1
        if self.grads_of(t):
            q.put(run)

    def scorer(self):  # rows_kernel's first issuing warp
        g = 0
        for it in range(self.items):
            if not (yield from self.wait("a_ready", self.a_ready, it)):
                return
            for _ in range(self.T):
                if not (yield from self.wait("full", self.full[g % self.stages], g // self.stages)):
                    return
                if g >= 2:
                    bar = self.r_full if self.slots else self.g_done
                    if not (yield from self.wait("buffer free", bar[g % 2], (g - 2) >> 1)):
                        return
                self.scores(it, g)
                g += 1

    def grader(self):  # its second
        g = 0
        for it in range(self.items):
            for t in range(self.T):
                if not (yield from self.wait("p_full", self.p_full[g % 8], g // 8)):
                    return
                self.grads(self.mma2, it, g, t, t == self.nkt)
                if not self.slots or self.grads_of(t):
                    self.mma2.put(self.g_done[self.where(g)].arrive)
                self.mma2.put(self.empty[g % self.stages].arrive)
                g += 1
            self.mma2.put(self.o_done.arrive)

    def issuer(self):  # cols_kernel's and dbias_kernel's
        for it in range(self.items):
            if not (yield from self.wait("a_ready", self.a_ready, it)):
                return
            for t in range(self.T + 2):
                g = it * self.T + t
                if t < self.T and not (yield from self.wait("full", self.full[g % self.stages], g // self.stages)):
                    return
                if t >= 2:
                    if not (yield from self.wait("p_full", self.p_full[(g - 2) % 8], (g - 2) // 8)):
                        return
                    self.grads(self.mma, it, g - 2, t - 2, t == 2)
                    self.mma.put(self.empty[(g - 2) % self.stages].arrive)
                if t < self.T:
                    self.scores(it, g)
            if self.kernel == "cols":
                self.mma.put(self.o_done.arrive)

    def group(self, w):
        ok, rows, dbias = True, self.kernel == "rows", self.kernel == "dbias"
        for it in range(self.items):
            if dbias:
                yield from self.meet("first meeting")
            if ok:
                self.kept[w].write(it, self.T)
                yield ("step", None)
                if dbias:
                    self.vectors[w].write(it, WARPGROUPS)
            self.a_ready.arrive()
            if dbias:
                yield from self.meet("second meeting")
            tiles = [t for t in range(self.T) if (it * self.T + t) % 2 == w]
            first = [t for t in tiles if rows and t < self.nkt]
            for part in (first, [t for t in tiles if t not in first]):
                for t in part:
                    g = it * self.T + t
                    ok = ok and (yield from self.wait("s_full", self.s_full[w], g >> 1))
                    ok = ok and (yield from self.wait("full (group)", self.full[g % self.stages], g // self.stages))
                    if not ok:
                        continue
                    if dbias:
                        assert all(v.tile == it for v in self.vectors) or not self.live, "row vectors of another chunk"
                    self.buf[w].read(g)
                    self.stage[g % self.stages].read(g)
                    if rows:
                        self.r_full[w].arrive()
                        yield ("step", None)
                    if self.grads_of(t):
                        n = it * self.nkt + t - self.nkt
                        if rows and self.slots and n >= 3:
                            ok = yield from self.wait("g_done", self.g_done[n % 3], n // 3 - 1)
                            if not ok:
                                break
                        self.slot[self.where(g)].write(g, 1)
                        yield ("step", None)
                    self.p_full[g % 8].arrive()
                if rows and part is first:
                    a = it % self.arrays
                    if ok:
                        self.joins[a, w].write(it, WARPGROUPS)
                    yield ("step", None)
                    yield from self.meet("join")
                    for o in range(WARPGROUPS):  # read one after the other
                        if ok:
                            self.joins[a, o].read(it)
                        yield ("step", None)
            if dbias:
                for v in self.vectors:
                    if ok:
                        v.read(it)
            else:
                ok = ok and (yield from self.wait("o_done", self.o_done, it))
                if ok:
                    assert self.acc_left == 0 or not self.live, "accumulators read before the last product"
                    self.acc.read(it)
                    yield ("step", None)

    # ---- scheduler
    def run(self, limit=400):
        """Every role to its end. A wait that stands for `limit` rounds in which nothing moves gives up and sets abort."""
        roles = [self.tma(), *(self.group(w) for w in range(WARPGROUPS))]
        roles += [self.scorer(), self.grader()] if self.kernel == "rows" else [self.issuer()]
        queues = [self.copies, self.mma, self.mma2]
        state = {}

        def advance(i, value=None):
            try:
                state[i] = roles[i].send(value)
            except StopIteration:
                state[i] = None
        for i in range(len(roles)):
            advance(i)
        speed = [self.rng.choice([1, 1, 5, 20]) for _ in roles]
        late = [self.rng.choice([1, 3, 20]) for _ in queues]
        idle = 0
        while any(s is not None for s in state.values()):
            moved = False
            for i in self.rng.sample(range(len(roles)), len(roles)):
                if state[i] is None or self.rng.randrange(speed[i]):
                    continue
                what, cond = state[i]
                if what == "step" or cond():
                    advance(i, True)
                elif what == "wait" and self.abort:
                    advance(i, False)
                else:
                    continue
                moved = True
            for q, every in zip(queues, late):
                if q.q and self.rng.randrange(every) == 0:
                    q.step()
                    moved = True
            idle = 0 if moved else idle + 1
            if idle > limit:
                waiting = [i for i, s in state.items() if s is not None and s[0] == "wait"]
                assert self.stall is not None and waiting and not self.abort, f"left waiting: roles {waiting}"
                self.abort, self.live, idle = True, False, 0
        # an issuing warp's last wait is for its own products, the copying thread's for its copies
        for q in queues:
            while q.q:
                q.step()
        assert self.met["n"] == 0, "a meeting with one side"
        return self.abort


CONFIGS = [("rows", True, 8), ("rows", True, 5), ("rows", False, 4), ("cols", False, 8), ("cols", False, 3),
           ("dbias", False, 5), ("dbias", False, 3)]
SIZES = [(1, 1), (3, 1), (2, 2), (4, 2), (3, 3), (2, 5), (1, 9)]


def sizes(kernel):
    # dbias_kernel's tiles come in pairs, one per buffer
    return [(i, n + n % 2 if kernel == "dbias" else n) for i, n in SIZES]


@pytest.mark.parametrize("kernel,slots,stages", CONFIGS)
def test_nothing_is_overwritten_between_items(kernel, slots, stages):
    for seed in range(60):
        for items, nkt in sizes(kernel):
            assert not Model(kernel, items, nkt, seed, slots, stages).run()


WAITS = {"rows": ["empty", "full", "a_ready", "buffer free", "s_full", "p_full", "join", "o_done"],
         "cols": ["empty", "full", "a_ready", "s_full", "p_full", "o_done"],
         # (dbias_kernel's second meeting is left out here: the row vectors are written
         # before a_ready, which every score waits for. It is what makes these plain
         # shared-memory writes visible, which a tensor-core commit in between need not.)
         "dbias": ["empty", "full", "a_ready", "s_full", "p_full", "first meeting"]}


def noticed(*args, **kw):
    n = 0
    for seed in range(40):
        for items, nkt in sizes(args[0]):
            try:
                Model(args[0], items, nkt, seed, *args[1:], **kw).run()
            except AssertionError:
                n += 1
    return n


@pytest.mark.parametrize("kernel,slots,stages,wait",
                         [(k, s, n, w) for k, s, n in [("rows", True, 5), ("rows", False, 4), ("cols", False, 8),
                                                       ("dbias", False, 5)]
                          for w in WAITS[k] + (["g_done"] if s else [])])
def test_every_wait_is_needed(kernel, slots, stages, wait):
    assert noticed(kernel, slots, stages, without=(wait,))


def test_one_join_array_is_a_race():
    # with one key tile a warpgroup can come to the next item's join while the
    # other still reads this one's: hence the two arrays, by the item's parity
    assert noticed("rows", True, 5, arrays=1)


@pytest.mark.parametrize("kernel,slots,stages", CONFIGS)
def test_all_roles_end_when_the_copies_stop(kernel, slots, stages):
    for seed in range(20):
        for items, nkt in sizes(kernel):
            tiles = items * (2 * nkt if kernel == "rows" else nkt)
            for stall in {0, min(1, tiles - 1), tiles // 2, tiles - 1}:
                assert Model(kernel, items, nkt, seed, slots, stages, stall=stall).run()
