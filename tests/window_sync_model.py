"""A host model of the warps, copies, products and barriers of the windowed attention kernel
(csrc/qmv_window_tc.cu, k_window_tc), on the simulator of attn_sync_model.

Beside the barriers' phases it keeps who holds what: a stream's scores, weights and output in
tensor memory and its queries in shared memory are written only when the last use has ended,
and read only when they are complete. Keyword arguments choose a protocol at fault."""
import random

from attn_sync_model import Barrier, Broken, Issuer, Ring, Sim


def window_tc(seed, segments, stages, two, apart=False, split=False, parted=False, copy=2000.0, slow=20.0,
              wait_ready=True, wait_done=True, one_barrier=False):
    """One block over segments, lists of steps that are true where values have to be looked at.

    stages: slots for keys and for values. wait_ready False: products wait for values that
    have come, not for those that have been looked at. wait_done False: with weights beside the
    scores, warps do not wait for the last products before they hand over new ones. one_barrier: both
    halves of a step's weights (split) arrive at the same barrier."""
    rng = random.Random(seed)
    sim = Sim(rng, slow)
    nq = 2 if two else 1
    kring, vring = Ring(sim, "keys'", stages[0], nq), Ring(sim, "values'", stages[1], nq)
    turns = two and not split and not apart
    B = lambda name, count: [Barrier(f"{name}[{s}]", count) for s in range(2)]  # noqa: E731
    q_full, q_empty, s_full, s_free, p_full, p_half, pv_done, o_full, turn = (
        B("q_full", 1), B("q_empty", 1), B("s_full", 1), B("s_free", 4), B("p_full", 4), B("p_half", 4),
        B("pv_done", 1), B("o_full", 1),
        B("turn", 1))
    if one_barrier:
        p_half = p_full
    vready = [Barrier(f"vready[{i}]", 1) for i in range(stages[1])]
    steps = [(k, i, i == len(seg) - 1, sp) for k, seg in enumerate(segments) for i, sp in enumerate(seg)]
    total = len(steps)
    streams = (lambda n: (0, 1)) if two else (lambda n: (n & 1,))
    unit = Issuer(sim)
    q_there, q_used = [None, None], [None, None]    # segment whose queries lie there, whose scores have ended
    s_holds, s_read = [None, None], [{}, {}]        # step of the scores, warps that have taken them
    o_taken, o_end = [{}, {}], [{}, {}]             # warps that have taken a segment's O; when products end
    p_written, h_written = [{}, {}], [{}, {}]       # warps' parts of a step's weights, of their first half
    scrubbed = {}

    def look(n):
        if n >= 0:
            yield vring.landed_wait(n)
            vring.read(n)
            yield sim.jitter(400 if steps[n][3] else 30)
            scrubbed[n] = 1
            sim.arrive(vready[n % stages[1]])

    def copier(ring):
        k = -1
        for n in range(total):
            if ring is vring and steps[n][1] == 0:
                k += 1
                for s in range(nq):
                    yield q_empty[s], k - 1
                    if k and q_used[s] != k - 1:
                        raise Broken(f"queries of segment {k} over those of {q_used[s]}")

                    def land(s=s, k=k):
                        q_there[s] = k
                        sim.arrive(q_full[s])
                    sim.at(sim.jitter(copy), land)
            yield ring.may_copy(n)
            ring.copy(n, copy)
            yield sim.jitter(60)
            if ring is vring:
                yield from look(n - 1)
        if ring is vring:
            yield from look(total - 1)

    def products(me):
        at = {"q": 0, "seen": -1, "o": 0, "fr": [0, 0], "f": [0, 0], "h": [0, 0], "t": 0}

        def peek():  # the keys of the next scores' step have come, and with them its flags
            n = at["q"]
            if at["seen"] != n:
                yield kring.landed_wait(n)
                kring.read(n)
                at["seen"] = n

        def scores_wait(s, again):
            n = at["q"]
            yield from peek()
            if steps[n][1] == 0:
                yield q_full[me], steps[n][0]
            if apart and again:
                yield s_free[s], at["fr"][s]
                at["fr"][s] += 1

        def scores_issue(s):
            n = at["q"]
            if q_there[me] != steps[n][0]:
                raise Broken(f"scores of segment {steps[n][0]} from queries of {q_there[me]}")
            kring.read(n)
            old = s_holds[s]
            if old is not None and s_read[s].get(old, 0) != 4:
                raise Broken(f"scores of step {n} over those of {old}, which are still read")
            if old is not None and not apart and (old not in o_end[s] or p_written[s].get(old, 0) != 4):
                raise Broken(f"scores of step {n} over the weights of {old}")
            s_holds[s] = n
            unit.product(256)
            unit.commit(s_full[s])

        def scores_done():
            n = at["q"]
            kring.release(n, unit)
            if steps[n][2]:
                unit.commit(q_empty[me], lambda: q_used.__setitem__(me, steps[n][0]))
            at["q"] += 1

        def scores(s, again):
            yield from scores_wait(s, again)
            scores_issue(s)
            scores_done()

        def output_wait(s):
            n = at["o"]
            yield (vready[n % stages[1]], n // stages[1]) if wait_ready else vring.landed_wait(n)
            if split:
                yield p_half[s], at["h"][s]
                at["h"][s] += 1
                if one_barrier:
                    at["f"][s] += 1
                if h_written[s].get(n, 0) != 4:
                    raise Broken(f"product of step {n} before the first half of its weights")
                unit.product(128)
            yield p_full[s], at["f"][s]
            at["f"][s] += 1
            if one_barrier:
                at["h"][s] += 1

        def output_issue(s, part):
            n = at["o"]
            k, i, _, special = steps[n]
            if part == 0:
                vring.read(n)
                if special and n not in scrubbed:
                    raise Broken(f"values of step {n} before they were looked at")
                if i < (1 if two else 2) and k and o_taken[s].get(k - 1, 0) != (4 if two else 8):
                    raise Broken(f"O of segment {k} over that of {k - 1}")
                if p_written[s].get(n, 0) != 4:
                    raise Broken(f"product of step {n} before its weights")
            unit.product(256)
            if split or apart:
                unit.commit(pv_done[s])

        def output_rest(s):
            if parted:
                yield p_full[s], at["f"][s]
                at["f"][s] += 1
                output_issue(s, 1)
            o_end[s][at["o"]] = unit.free

        def output_done(s):
            n = at["o"]
            vring.release(n, unit)
            if steps[n][2]:
                unit.commit(o_full[s])
                if not two:
                    unit.commit(o_full[s ^ 1])
            at["o"] += 1

        def output(s):
            yield from output_wait(s)
            output_issue(s, 0)
            yield from output_rest(s)
            output_done(s)

        starts = lambda: at["q"] < total and steps[at["q"]][1] == 0  # noqa: E731
        if turns:
            yield from scores(me, False)
            for n in range(total):
                more = n + 1 < total
                if more:
                    yield from peek()
                held = more and starts()
                now = more and not held
                if now:
                    yield from scores_wait(me, True)
                yield from output_wait(me)
                if me or n:
                    yield turn[me], at["t"]
                    at["t"] += 1
                output_issue(me, 0)
                yield from output_rest(me)
                if now:
                    scores_issue(me)
                sim.arrive(turn[me ^ 1])
                output_done(me)
                if now:
                    scores_done()
                if held:
                    yield from scores(me, True)
                yield sim.jitter(20)
        elif two:
            yield from scores(me, False)
            for n in range(total):
                if apart and n + 1 < total:
                    yield from scores(me, True)
                yield from output(me)
                if not apart and n + 1 < total:
                    yield from scores(me, True)
                yield sim.jitter(20)
        else:
            def ahead(upto):
                while at["q"] < total and at["q"] < upto:
                    yield from scores(at["q"] & 1, at["q"] >= 2)
            yield from ahead(1)
            if total > 1:
                yield from peek()
                if not starts():
                    yield from ahead(2)
            for n in range(total):
                if apart and at["q"] == n + 2 and at["q"] < total:
                    yield from peek()
                    if not starts():
                        yield from ahead(n + 3)
                yield from ahead(n + 1)
                yield from output(n & 1)
                yield from ahead(n + 2)
                if at["q"] < total:
                    yield from peek()
                    if not starts():
                        yield from ahead(n + 3)
                yield sim.jitter(20)

    def softmax(s, w):
        sp = op = vp = 0
        again, n, last = False, 0, None
        for k, seg in enumerate(segments):
            mine = []
            for i in range(len(seg)):
                if s in streams(n + i):
                    mine.append((n + i, seg[i]))
            yield sim.jitter(50)
            for x, special in mine:
                yield s_full[s], sp
                sp += 1
                if s_holds[s] != x:
                    raise Broken(f"softmax of step {x} reads scores of {s_holds[s]}")
                yield sim.jitter(150)
                s_read[s][x] = s_read[s].get(x, 0) + 1
                if apart:
                    sim.arrive(s_free[s])
                    if again and wait_done:
                        yield pv_done[s], vp
                        vp += 1
                if last is not None and sim.now < o_end[s].get(last, float("inf")):
                    raise Broken(f"step {x} moves O or writes weights before the products of {last} end")
                if split:
                    yield sim.jitter(300)
                    h_written[s][x] = h_written[s].get(x, 0) + 1
                    sim.arrive(p_half[s])
                yield sim.jitter(300 if split else 600)
                p_written[s][x] = p_written[s].get(x, 0) + 1
                if not split:
                    sim.arrive(p_full[s])
                else:
                    for _ in range(2 if parted else 1):
                        sim.arrive(p_full[s])
                        yield pv_done[s], vp
                        vp += 1
                        yield sim.jitter(150)
                again, last = True, x
            n += len(seg)
            yield o_full[s], op
            op += 1
            if not two:
                yield pairs[w], 2
            for z in (s,) if two else (0, 1):
                for x in range(n - len(seg), n):
                    if z in streams(x) and sim.now < o_end[z].get(x, float("inf")):
                        raise Broken(f"O of segment {k} is read before step {x} ends")
            yield sim.jitter(500)
            for z in (s,) if two else (0, 1):
                o_taken[z][k] = o_taken[z].get(k, 0) + 1
            if not two:
                yield pairs[w], 2

    pairs = [[] for _ in range(4)]
    sim.start("key copies", copier(kring))
    sim.start("value copies", copier(vring))
    for s in range(nq):
        sim.start(f"products {s}", products(s))
    for s in range(2):
        for w in range(4):
            sim.start(f"softmax {s}.{w}", softmax(s, w))
    sim.run()
