"""A host model of the warps, copies, products and barriers of the tcgen05 attention kernels.

Every warp is a generator that yields what it waits for; the times of copies, products
and steps are drawn. A barrier knows how many of its phases are complete, and a wait
is the hardware's: it passes when the phase's parity says so. Each wait also carries
the phase that it means, so that one which passes for another phase, a slot that is
copied into before its last use, or a table that is read too late raises Broken.

`attn_tc` follows csrc/qmv_attn_tc.cu (k_attn_tc), `weights_tc` csrc/qmv_attn_weights.cu
(k_weights_tc). Their keyword arguments can choose a protocol that was found wanting,
which the model has to notice.
"""
import heapq
import random


class Broken(Exception):
    pass


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.done, self.waiting = name, count, count, 0, []


class Sim:
    """Events in time; actors are generators that yield a delay (a number), (barrier,
    phase) for a wait, or (named, n) with a list for a barrier of n warps."""

    def __init__(self, rng, slow=1.0):
        self.rng, self.now, self.heap, self.n, self.alive, self.slow = rng, 0.0, [], 0, 0, slow
        self.names = {}

    def at(self, delay, f):
        self.n += 1
        heapq.heappush(self.heap, (self.now + delay, self.n, f))

    def start(self, name, gen):
        self.alive += 1
        self.names[gen] = name
        self.step(gen)

    def step(self, gen):
        try:
            what = next(gen)
        except StopIteration:
            self.alive -= 1
            del self.names[gen]
            return
        if isinstance(what, (int, float)):
            self.at(what, lambda: self.step(gen))
        elif isinstance(what[0], Barrier):
            self.poll(gen, *what)
        else:
            crowd, n = what
            crowd.append(gen)
            if len(crowd) == n:
                for g in crowd:
                    self.at(self.jitter(10), lambda g=g: self.step(g))
                crowd.clear()

    def poll(self, gen, bar, phase):
        if (bar.done & 1) == (phase & 1):       # not complete, as far as the parity tells
            bar.waiting.append((gen, phase))
        elif bar.done != phase + 1:
            raise Broken(f"{self.names[gen]} waits for phase {phase} of {bar.name}, "
                         f"which passes with {bar.done} complete")
        else:
            self.at(self.jitter(5), lambda: self.step(gen))

    def arrive(self, bar):
        bar.left -= 1
        if bar.left == 0:
            bar.left = bar.count
            bar.done += 1
            for gen, phase in bar.waiting:
                self.at(self.jitter(20), lambda gen=gen, phase=phase: self.poll(gen, bar, phase))
            bar.waiting = []

    def jitter(self, mean):
        """Mostly near the mean, now and then much later."""
        t = mean * self.rng.uniform(0.5, 1.5)
        if self.rng.random() < 0.05:
            t += mean * self.slow * self.rng.expovariate(1.0)
        return t

    def run(self):
        while self.heap:
            self.now, _, f = heapq.heappop(self.heap)
            f()
        if self.alive:
            raise Broken("stuck: " + ", ".join(sorted(self.names.values())))


class Issuer:
    """A thread's products: they end in order, and a commit arrives after those before it."""

    def __init__(self, sim):
        self.sim, self.free = sim, 0.0

    def product(self, mean):
        self.free = max(self.free, self.sim.now) + self.sim.jitter(mean)

    def commit(self, bar, then=None):
        self.free = max(self.free, self.sim.now)

        def land():
            if then:
                then()
            self.sim.arrive(bar)
        self.sim.at(self.free - self.sim.now, land)


class Ring:
    """Slots of copied tiles: entry e lies in slot e % stages."""

    def __init__(self, sim, name, stages, readers):
        self.sim, self.stages, self.readers = sim, stages, readers
        self.full = [Barrier(f"{name} full[{i}]", 1) for i in range(stages)]
        self.empty = [Barrier(f"{name} empty[{i}]", readers) for i in range(stages)]
        self.issued, self.landed, self.used = [None] * stages, [None] * stages, {}

    def may_copy(self, e):
        return self.empty[e % self.stages], e // self.stages - 1

    def copy(self, e, mean):
        i = e % self.stages
        last = self.issued[i]
        if last != (e - self.stages if e >= self.stages else None):
            raise Broken(f"entry {e} is copied over entry {last}")
        if last is not None and self.used.get(last, 0) != self.readers:
            raise Broken(f"entry {e} is copied over entry {last}, which is in use")
        self.issued[i] = e

        def land():
            self.landed[i] = e
            self.sim.arrive(self.full[i])
        self.sim.at(self.sim.jitter(mean), land)

    def landed_wait(self, e):
        return self.full[e % self.stages], e // self.stages

    def read(self, e):
        if self.landed[e % self.stages] != e:
            raise Broken(f"entry {e} is read, its slot holds {self.landed[e % self.stages]}")

    def release(self, e, issuer):
        def then():
            self.used[e] = self.used.get(e, 0) + 1
        issuer.commit(self.empty[e % self.stages], then)


def attn_tc(seed, segments, stages, two, apart=False, split=False, parted=False, copy=2000.0,
            slow=20.0, rings=2, ack=True):
    """One block of k_attn_tc over segments of the given numbers of key tiles.

    stages: slots for keys and for values; two: both streams take every tile (more than
    128 rows); apart: weights beside the scores (64-element heads); split, parted: fp32
    outputs, O in two halves. rings 1: keys and values by turns in one ring of both's
    slots, in the order of the products. ack False: a stream without tiles in a segment
    does not answer."""
    rng = random.Random(seed)
    sim = Sim(rng, slow)
    readers = 2 if two else 1
    if rings == 2:
        kring, vring = Ring(sim, "keys'", stages[0], readers), Ring(sim, "values'", stages[1], readers)
    else:
        kring = vring = Ring(sim, "the ring's", sum(stages), readers)
    lag = 1 if two else 2  # tiles a product P V runs behind its scores
    step = 1 if two else 2
    B = lambda name, count: [Barrier(f"{name}[{s}]", count) for s in range(2)]
    s_full, p_ready, o_full, s_free, turn, pv_done = (
        B("s_full", 1), B("p_ready", 4), B("o_full", 1), B("s_free", 4), B("turn", 4), B("pv_done", 1))
    q_full = Barrier("q_full", 8)
    tiles = {"n": None}
    crowd = []

    # a tile's entry; base: the tiles of the segments before
    def entry_k(base, t, n):
        if rings == 2:
            return base + t
        return 2 * base + (t if t < lag else 2 * t + (0 if apart else 1) - lag)

    def entry_v(base, t, n):
        if rings == 2:
            return base + t
        return 2 * base + min(t + lag + (1 if apart else 0), n) + t

    def copier(ring, entry):
        base = 0
        for n in segments:
            for t in range(n):
                e = entry(base, t, n)
                yield ring.may_copy(e)
                ring.copy(e, copy)
                yield sim.jitter(60)
            base += n
            yield sim.jitter(300)

    def products(s):
        unit = Issuer(sim)
        base = fp = pp = 0

        def scores(t, n):
            e = entry_k(base, t, n)
            yield kring.landed_wait(e)
            kring.read(e)
            unit.product(256)
            unit.commit(s_full[s])
            kring.release(e, unit)

        for k, n in enumerate(segments):
            yield q_full, k
            if tiles["n"] != (k, n):
                raise Broken(f"products {s} of segment {k} read the tiles of {tiles['n']}")
            t0 = 0 if two else s
            if t0 < n:
                yield from scores(t0, n)
            for t in range(t0, n, step):
                if apart and t + step < n:
                    yield s_free[s], fp
                    fp += 1
                    yield from scores(t + step, n)
                e = entry_v(base, t, n)
                if two:
                    yield vring.landed_wait(e)
                yield p_ready[s], pp
                if not two:
                    yield vring.landed_wait(e)
                pp += 1
                vring.read(e)
                unit.product(256)
                if parted:
                    unit.commit(pv_done[s])
                    yield p_ready[s], pp
                    pp += 1
                    unit.product(256)
                vring.release(e, unit)
                if apart or split:
                    unit.commit(pv_done[s])
                if t + step >= n:
                    unit.commit(o_full[s])
                elif not apart:
                    yield from scores(t + step, n)
                yield sim.jitter(20)
            if apart and t0 < n:
                yield s_free[s], fp
                fp += 1
            if ack and t0 >= n:
                sim.arrive(o_full[s])
            base += n

    def softmax(s, w):
        base = sp = op = tp = vp = 0
        for k, n in enumerate(segments):
            ns = n if two else (n + 1 - s) // 2
            yield sim.jitter(400)                     # queries
            if s == 0 and w == 0:
                tiles["n"] = (k, n)
            sim.arrive(q_full)
            yield crowd, 8
            for i in range(ns):
                t = i if two else 2 * i + s
                yield s_full[s], sp
                sp += 1
                if i > 0 or s > 0:
                    yield turn[s], tp + (i if s else i - 1)
                if (not two or s == 0) and (t == n - 1 or rng.random() < 0.2):  # values looked at
                    e = entry_v(base, t, n)
                    yield vring.landed_wait(e)
                    vring.read(e)
                    yield sim.jitter(300)
                if apart:
                    sim.arrive(turn[s ^ 1])
                    sim.arrive(s_free[s])
                    if i > 0:
                        yield pv_done[s], vp
                        vp += 1
                yield sim.jitter(1000)
                if not apart:
                    sim.arrive(turn[s ^ 1])
                sim.arrive(p_ready[s])
                if split:
                    yield pv_done[s], vp
                    vp += 1
                    if parted:
                        sim.arrive(p_ready[s])
                        yield pv_done[s], vp
                        vp += 1
            if ns > 0 or ack:
                yield o_full[s], op
                op += 1
            if apart and ns > 0:
                vp += 1
            yield crowd, 8
            yield sim.jitter(500)
            yield crowd, 8
            tp += n if two else (n + s) // 2
            base += n

    sim.start("copies of keys", copier(kring, entry_k))
    sim.start("copies of values", copier(vring, entry_v))
    for s in range(2):
        sim.start(f"products {s}", products(s))
        for w in range(4):
            sim.start(f"softmax {s}.{w}", softmax(s, w))
    sim.run()


def weights_tc(seed, segments, stages, copy=2000.0, slow=20.0, own_buffers=True):
    """One block of k_weights_tc over segments of (key tiles, row tiles).

    own_buffers False: score buffers in the order of all products, whichever group takes
    them."""
    rng = random.Random(seed)
    sim = Sim(rng, slow)
    ring = Ring(sim, "keys'", stages, 1)
    s_full = [Barrier(f"s_full[{i}]", 1) for i in range(4)]
    s_free = [Barrier(f"s_free[{i}]", 4) for i in range(4)]
    held = [None] * 4
    q_full = Barrier("q_full", 8)
    tables = {}
    crowd = []
    units = sum(n for n, _ in segments)

    def place(group, mine, job):
        return (2 * group + (mine & 1), mine >> 1) if own_buffers else (job & 3, job >> 2)

    def copier(first):
        for x in range(first, units, 2):
            yield ring.may_copy(x)
            ring.copy(x, copy)
            yield sim.jitter(60)

    def products():
        unit = Issuer(sim)
        x = job = 0
        count = [0, 0]
        for k, (n, nq) in enumerate(segments):
            yield q_full, k
            if tables.get("now") != (k, n, nq):
                raise Broken(f"products of segment {k} read the tables of {tables.get('now')}")
            for t in range(n):
                yield ring.landed_wait(x)
                ring.read(x)
                for _ in range(nq):
                    buf, phase = place(t & 1, count[t & 1], job)
                    if phase > 0:
                        yield s_free[buf], phase - 1
                    if held[buf] is not None:
                        raise Broken(f"scores {held[buf]} are overwritten in use")
                    held[buf] = job
                    unit.product(256)
                    unit.commit(s_full[buf])
                    count[t & 1] += 1
                    job += 1
                    yield sim.jitter(20)
                ring.release(x, unit)
                x += 1

    def softmax(s, w):
        job0 = mine = 0
        for k, (n, nq) in enumerate(segments):
            yield sim.jitter(400)
            if s == 0 and w == 0:
                tables["now"] = (k, n, nq)
            sim.arrive(q_full)
            yield crowd, 8
            for t in range(s, n, 2):
                yield sim.jitter(50)
                for r in range(nq):
                    job = job0 + t * nq + r
                    buf, phase = place(s, mine, job)
                    yield s_full[buf], phase
                    if held[buf] != job:
                        raise Broken(f"scores {job} are read, the buffer holds {held[buf]}")
                    yield sim.jitter(600)
                    mine += 1
                    # (the warps' reads end together with the last arrival)
                    if s_free[buf].left == 1:
                        held[buf] = None
                    sim.arrive(s_free[buf])
            yield crowd, 8
            job0 += n * nq

    for first in range(2):
        sim.start(f"copies {first}", copier(first))
    sim.start("products", products())
    for s in range(2):
        for w in range(4):
            sim.start(f"softmax {s}.{w}", softmax(s, w))
    sim.run()
