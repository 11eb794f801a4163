"""The barriers of qr_kernel and qp_kernel, attention over pages of 8-bit codes, modelled on the CPU.

As in test_paged_protocol_cpu.py: every warp is a generator that yields the barrier phase it waits for, copies and the commits of MMAs are events
that come later, and all run in random order.  What shared and tensor memory hold is modelled as the number of the tile (or half, or item) that was
written there last, and checked where it is read.  A run may be given up at any moment: from then on a wait that is not over may fail, and it need
not, as the copies and MMAs still under way come in.  All warps have to leave, and the end of the kernel has to wait for everything that is still
under way.
"""

import itertools
import random

import pytest
from test_paged_protocol_cpu import JOBS, Bar


class Base:
    drains = True  # warps that issue MMAs wait for their last commits

    def __init__(self, jobs, rng):
        self.jobs, self.rng, self.slot, self.up = jobs, rng, [None] * JOBS, False
        self.job_full = self.bars("job_full", JOBS, 1)
        self.later = {}

    def bars(self, name, n, count):
        return [Bar(name + str(i), count) for i in range(n)]

    def each_job(self):
        """Yields waits, then ("job", its number, record); ends behind the last one."""
        for at in itertools.count():
            yield self.job_full[at % JOBS], at // JOBS
            job = self.slot[at % JOBS]
            self.job_empty[at % JOBS].arrive()
            if job is None:
                return
            yield "job", at, job

    def over_jobs(self, body):
        for step in self.each_job():
            if step[0] == "job":
                yield from body(step[1], step[2])
            else:
                yield step

    def post_jobs(self, body):
        for at, job in enumerate(self.jobs + [None]):
            if at >= JOBS:
                yield self.job_empty[at % JOBS], at // JOBS - 1
            self.slot[at % JOBS] = job
            self.job_full[at % JOBS].arrive()
            if job is not None:
                yield from body(job)

    # a wait that nothing but its barrier ends
    def bound(self, wait):
        return False

    # a warp that goes on with a wait given up
    def stays(self, role):
        return False

    def expect(self, holds, what=""):
        """What memory holds is nobody's business once the run is given up."""
        assert holds or self.up, what

    def happen(self, name):
        events = self.later[name]
        events.pop(0 if name.startswith("MMA") else self.rng.randrange(len(events)))()

    def run(self, moves=None):
        """moves: given up after so many."""
        roles = self.roles()
        waits = dict.fromkeys(roles)
        speed = {k: self.rng.choice([1, 1, 5, 20]) for k in list(roles) + ["later " + k for k in self.later]}
        def go(k, lost=None):
            try:
                waits[k] = roles[k].send(lost)
            except StopIteration:
                del roles[k]

        while roles:
            self.up = moves is not None and moves <= 0
            able = [k for k in roles if waits[k] is None or waits[k][0].over(waits[k][1])]
            failing = ["fail " + k for k in roles if self.up and k not in able and not self.bound(waits[k])]
            choice = able + failing + ["later " + k for k, events in self.later.items() if events]
            assert choice, "%s: %s" % ("hang" if self.up else "deadlock", {k: (waits[k][0].name, waits[k][0].done, waits[k][1]) for k in roles})
            k = self.rng.choices(choice, [speed.get(a, 3) for a in choice])[0]
            moves = None if moves is None else moves - 1
            if k.startswith("later "):
                self.happen(k[6:])
            elif k.startswith("fail ") and not self.stays(k[5:]):
                del roles[k[5:]]
            elif k.startswith("fail "):
                go(k[5:], True)
            else:
                go(k)
        if moves is not None:
            self.drain()
        assert not any(self.later.values()), "still under way at the end: %s" % {k: len(v) for k, v in self.later.items() if v}

    def drain(self):
        for name in self.later:
            while name.startswith("MMA") and self.later[name]:
                self.happen(name)
        for name, full, loads in self.loads():
            for i in range(min(loads, len(full))):
                at = loads - 1 - i
                while full[at % len(full)].done <= at // len(full):
                    assert self.later[name], "the end waits for a copy that nobody asked for"
                    self.happen(name)


class Few(Base):
    """qr_kernel: a loading warp, one of MMAs, four of softmax that meet once an item, a tile, an item's end and at their end, at a named barrier,
    which no limit ends.  A wait given up is told at the next item's first meeting."""

    together = True  # a softmax warp whose wait is given up comes to the meetings that the others are on their way to

    def __init__(self, jobs, stages, rng):
        super().__init__(jobs, rng)
        self.stages, self.scales = stages, stages + 2
        self.job_empty = self.bars("job_empty", JOBS, 5)
        self.k_full, self.k_empty, self.v_full, self.v_empty = (self.bars(n, stages, 1) for n in ("k_full", "k_empty", "v_full", "v_empty"))
        self.sc_full = self.bars("sc_full", self.scales, 1)
        self.s_full, self.s_free, self.p_ready, self.o_full, self.q_ready, self.meet = (
            Bar(n, c) for n, c in (("s_full", 1), ("s_free", 4), ("p_ready", 4), ("o_full", 1), ("q_ready", 4), ("meet", 4)))
        self.drained = Bar("drained", 1)
        self.later = {"K": [], "V": [], "MMA": []}
        self.k, self.v, self.sc = [None] * stages, [None] * stages, [None] * self.scales
        self.q, self.p, self.top, self.s, self.o = [None] * 4, [None] * 4, [[None] * 4, [None] * 4], None, None
        self.k_loads = self.v_loads = 0
        self.said = {}  # at each meeting that tells

    def bound(self, wait):
        return wait[0] is self.meet

    def stays(self, role):
        return self.together and role.startswith("soft")

    def loads(self):
        return ("K", self.k_full, self.k_loads), ("V", self.v_full, self.v_loads)

    def roles(self):
        return {"load": self.loader(), "mma": self.mma(), **{"soft%d" % w: self.softmax(w) for w in range(4)}}

    def loader(self):
        def body(job):
            for t in range(job["n"] + 1):
                if t < job["n"]:
                    at = self.k_loads
                    slot, turn = at % self.stages, at // self.stages
                    if turn > 0:
                        yield self.k_empty[slot], turn - 1
                    self.sc[at % self.scales] = at
                    self.sc_full[at % self.scales].arrive()

                    def land(slot=slot, at=at):
                        self.k[slot] = at
                        self.k_full[slot].arrive()

                    self.later["K"].append(land)
                    self.k_loads += 1
                    yield None
                if t > 0:
                    at = self.v_loads
                    slot, turn = at % self.stages, at // self.stages
                    if turn > 0:
                        yield self.v_empty[slot], turn - 1

                    def land(slot=slot, at=at):
                        self.v[slot] = at
                        self.v_full[slot].arrive()

                    self.later["V"].append(land)
                    self.v_loads += 1
                    yield None

        return self.post_jobs(body)

    def mma(self):
        g = 0
        commit = self.later["MMA"].append

        def score(i, item):
            slot = i % self.stages
            yield self.k_full[slot], i // self.stages
            if i > 0:
                yield self.s_free, i - 1

            def make():
                self.expect(self.k[slot] == i and self.q == [item] * 4)
                self.s = i
                self.s_full.arrive()

            commit(make)
            commit(self.k_empty[slot].arrive)

        def body(item, job):
            nonlocal g
            n = job["n"]
            yield self.q_ready, item
            yield from score(g, item)
            for i in range(g, g + n):
                if i + 1 < g + n:
                    yield from score(i + 1, item)
                slot = i % self.stages
                yield self.v_full[slot], i // self.stages
                yield self.p_ready, i

                def make(i=i, slot=slot):
                    self.expect(self.v[slot] == i and self.p == [i] * 4)
                    self.o = i
                    self.o_full.arrive()

                commit(make)
                commit(self.v_empty[slot].arrive)
            g += n

        yield from self.over_jobs(body)
        if self.drains:
            commit(self.drained.arrive)
            yield self.drained, 0

    def softmax(self, w):
        g = met = 0  # tiles, meetings

        def meet(said=None):
            nonlocal met
            kind, all_said = self.said.setdefault(met, (said is None, []))
            assert kind == (said is None), "warps at one barrier wait in two ways"
            all_said.append(said)
            self.meet.arrive()
            met += 1
            return self.meet, met - 1

        for item in itertools.count():
            lost = yield self.job_full[item % JOBS], item // JOBS
            job = None
            if not lost:
                job = self.slot[item % JOBS]
                self.job_empty[item % JOBS].arrive()
            if job is None:
                break
            n = job["n"]
            self.expect(not [e for e in self.later["MMA"] if e.__name__ == "make"], "q's terms are written while an MMA reads them")
            self.q[w] = item
            self.q_ready.arrive()
            yield meet(True)
            if not all(self.said[met - 1][1]):
                return
            for i in range(n):
                owed = n - i + 1
                lost = yield self.sc_full[g % self.scales], g // self.scales
                if lost:
                    break
                self.expect(self.sc[g % self.scales] == g)
                lost = yield self.s_full, g
                if lost:
                    break
                self.expect(self.s == g)
                yield None
                self.expect(self.s == g)
                self.s_free.arrive()
                self.top[i & 1][w] = g
                yield meet()
                owed -= 1
                self.expect(self.top[i & 1] == [g] * 4)
                yield None
                self.expect(self.top[i & 1] == [g] * 4)
                if i + 1 == n and job["tail"]:
                    lost = yield self.v_full[g % self.stages], g // self.stages
                    if lost:
                        break
                    self.expect(self.v[g % self.stages] == g)
                if i > 0:
                    lost = yield self.o_full, g - 1
                    if lost:
                        break
                    self.expect(self.o == g - 1)
                    yield None
                    self.expect(self.o == g - 1)
                self.p[w] = g
                self.p_ready.arrive()
                g += 1
            if not lost:
                owed = 1
                lost = yield self.o_full, g - 1
            if lost:
                for _ in range(owed):
                    yield meet()
                break
            self.expect(self.o == g - 1)
            yield None
            self.expect(self.o == g - 1)
            self.top[n & 1][w] = "sums", item
            yield meet()
            self.expect(self.top[n & 1] == [("sums", item)] * 4)
            yield None
            self.expect(self.top[n & 1] == [("sums", item)] * 4)
        yield meet(not lost)


class Many(Base):
    """qp_kernel: a loading warp, one of MMAs for each stream, four that convert V, four of softmax for each stream, which take S in halves."""

    late_scales = 0  # scales' places beside those that the kernel has

    def __init__(self, jobs, bf16, rng):
        super().__init__(jobs, rng)
        self.stages, self.codes, self.wide = (3, 2, 2) if bf16 else (2, 1, 2)
        self.scales = self.stages + 2 + self.late_scales
        self.job_empty = self.bars("job_empty", JOBS, 14)
        self.k_full, self.k_empty = self.bars("k_full", self.stages, 1), self.bars("k_empty", self.stages, 2)
        self.c_full, self.c_empty = self.bars("c_full", self.codes, 1), self.bars("c_empty", self.codes, 4)
        self.v_full, self.v_empty = self.bars("v_full", self.wide, 4), self.bars("v_empty", self.wide, 2)
        self.sc_full = self.bars("sc_full", self.scales, 1)
        self.s_full, self.p_ready, self.o_step = ([self.bars("%s%d" % (n, d), 2, c) for d in range(2)] for n, c in (("s_full", 1), ("p_ready", 4), ("o_step", 1)))
        self.q_ready = self.bars("q_ready", 2, 4)
        self.drained = self.bars("drained", 2, 1)
        self.later = {"K": [], "C": [], "MMA0": [], "MMA1": []}
        self.k, self.c, self.sc = [None] * self.stages, [None] * self.codes, [None] * self.scales
        self.v = [[None] * 4 for _ in range(self.wide)]
        self.q = [[None] * 4 for _ in range(2)]
        self.sp = [[[None] * 4 for _ in range(2)] for _ in range(2)]  # S or P of a stream's half, by warp's rows
        self.o = [-1, -1]  # halves that O has
        self.k_loads = self.c_loads = 0

    def loads(self):
        return ("K", self.k_full, self.k_loads), ("C", self.c_full, self.c_loads)

    def roles(self):
        return {"load": self.loader(), **{"mma%d" % d: self.mma(d) for d in range(2)}, **{"turn%d" % c: self.convert(c) for c in range(4)},
                **{"soft%d%d" % (d, w): self.softmax(d, w) for d in range(2) for w in range(4)}}

    def loader(self):
        def body(job):
            for t in range(job["n"] + 1):
                if t < job["n"]:
                    at = self.k_loads
                    slot, turn = at % self.stages, at // self.stages
                    if turn > 0:
                        yield self.k_empty[slot], turn - 1
                    self.sc[at % self.scales] = at
                    self.sc_full[at % self.scales].arrive()

                    def land(slot=slot, at=at):
                        self.k[slot] = at
                        self.k_full[slot].arrive()

                    self.later["K"].append(land)
                    self.k_loads += 1
                    yield None
                if t > 0:
                    at = self.c_loads
                    slot, turn = at % self.codes, at // self.codes
                    if turn > 0:
                        yield self.c_empty[slot], turn - 1

                    def land(slot=slot, at=at):
                        self.c[slot] = at
                        self.c_full[slot].arrive()

                    self.later["C"].append(land)
                    self.c_loads += 1
                    yield None

        return self.post_jobs(body)

    def mma(self, d):
        g = mine = items = 0
        commit = self.later["MMA%d" % d].append

        def score(i, b, tile, item):
            slot = i % self.stages
            if b == 0:
                yield self.k_full[slot], i // self.stages

            def make():
                self.expect(self.k[slot] == i and self.q[d] == [item] * 4)
                self.sp[d][b] = [("S", 2 * tile + b)] * 4
                self.s_full[d][b].arrive()

            commit(make)
            if b == 1:
                commit(self.k_empty[slot].arrive)

        def body(_, job):
            nonlocal g, mine, items
            n = job["n"]
            if d == 1 and not job["both"]:
                for i in range(g, g + n):
                    yield self.k_full[i % self.stages], i // self.stages
                    self.k_empty[i % self.stages].arrive()
                    yield self.v_full[i % self.wide], i // self.wide
                    self.v_empty[i % self.wide].arrive()
                g += n
                return
            item = items
            yield self.q_ready[d], item
            items += 1
            for b in range(2):
                yield from score(g, b, mine, item)
            for i in range(g, g + n):
                slot = i % self.wide
                yield self.v_full[slot], i // self.wide
                for b in range(2):
                    yield self.p_ready[d][b], mine

                    def make(b=b, half=2 * mine + b, slot=slot, i=i):
                        self.expect(self.v[slot] == [i] * 4 and self.sp[d][b] == [("P", half)] * 4)
                        self.o[d] = half
                        self.o_step[d][b].arrive()

                    commit(make)
                    if b == 1:
                        commit(self.v_empty[slot].arrive)
                    if i + 1 < g + n:
                        yield from score(i + 1, b, mine + 1, item)
                mine += 1
            g += n

        yield from self.over_jobs(body)
        if self.drains:
            commit(self.drained[d].arrive)
            yield self.drained[d], 0

    def convert(self, c):
        g = 0

        def body(_, job):
            nonlocal g
            for _ in range(job["n"]):
                a, to = g % self.codes, g % self.wide
                yield self.c_full[a], g // self.codes
                if g >= self.wide:
                    yield self.v_empty[to], g // self.wide - 1
                self.expect(self.c[a] == g and self.sc[g % self.scales] == g)
                yield None
                self.expect(self.c[a] == g and self.sc[g % self.scales] == g)
                self.v[to][c] = g
                self.c_empty[a].arrive()
                self.v_full[to].arrive()
                g += 1

        return self.over_jobs(body)

    def softmax(self, d, w):
        g = mine = items = 0

        def body(_, job):
            nonlocal g, mine, items
            n = job["n"]
            if d == 1 and not job["both"]:
                g += n
                return
            # what an MMA has yet to read of the item before: q's terms, and O by what takes its place
            self.expect(not [e for e in self.later["MMA%d" % d] if e.__name__ == "make"], "q's terms are written while an MMA reads them")
            self.q[d][w] = items
            items += 1
            self.q_ready[d].arrive()
            for i in range(2 * n):
                b, tile = i & 1, g + i // 2
                if b == 0:
                    yield self.sc_full[tile % self.scales], tile // self.scales
                yield self.s_full[d][b], mine >> 1
                self.expect(self.sc[tile % self.scales] == tile and self.sp[d][b][w] == ("S", mine))
                yield None
                self.expect(self.sc[tile % self.scales] == tile and self.sp[d][b][w] == ("S", mine))
                if i > 0 and self.rng.random() < 0.3:  # the reference grew: O is rescaled
                    yield self.o_step[d][b ^ 1], (mine - 1) >> 1
                    self.expect(self.o[d] == mine - 1)
                    yield None
                    self.expect(self.o[d] == mine - 1)
                self.sp[d][b][w] = "P", mine
                self.p_ready[d][b].arrive()
                mine += 1
            g += n
            yield self.o_step[d][0], (mine - 2) >> 1
            yield self.o_step[d][1], (mine - 1) >> 1
            self.expect(self.o[d] == mine - 1)
            yield None
            self.expect(self.o[d] == mine - 1)

        return self.over_jobs(body)


def _jobs(rng, most):
    return [{"n": rng.choice([1, 1, 1, 2, 2, 3, 4, 5, 9]), "tail": rng.random() < 0.5, "both": rng.random() < 0.6} for _ in range(rng.randint(1, most))]


def _make(kind, seed, most):
    rng = random.Random(seed)
    jobs = _jobs(rng, most)
    if kind == "many":
        return Many(jobs, seed % 2 == 0, rng), rng
    return Few(jobs, rng.choice([2, 3, 4, 6]), rng), rng


@pytest.mark.parametrize("kind", ["few", "many"])
def test_roles_keep_in_step(kind):
    for seed in range(250):
        _make(kind, seed, 20)[0].run()


@pytest.mark.parametrize("kind", ["few", "many"])
def test_a_run_that_is_given_up_ends_with_nothing_under_way(kind):
    for seed in range(1000):
        run, rng = _make(kind, seed, 8)
        run.run(int(2 ** rng.uniform(0, 9)))


@pytest.mark.parametrize("mistake", ["leaves at once", "leaves its item at once", "tells nobody"])
def test_the_model_sees_what_a_softmax_warp_owes(mistake):
    """A warp that leaves where its wait is given up: another one, whose wait was over, waits at the named barrier for ever."""

    class Wrong(Few):
        together = mistake != "leaves at once"

        def softmax(self, w):
            role, lost, left = super().softmax(w), None, False
            while True:
                try:
                    step = role.send(lost)
                except StopIteration:
                    return
                index = step[1] if step is not None and step[0] is self.meet else None
                if index is not None and left and mistake == "leaves its item at once" and self.said[index][0]:
                    return
                if index is not None and mistake == "tells nobody" and self.said[index][1] and self.said[index][1][-1] is False:
                    self.said[index][1][-1] = True
                lost = yield step
                left = left or bool(lost)

    with pytest.raises(AssertionError, match="hang"):
        for seed in range(1000):
            rng = random.Random(seed)
            Wrong(_jobs(rng, 8), rng.choice([2, 3, 4, 6]), rng).run(int(2 ** rng.uniform(0, 9)))


@pytest.mark.parametrize("kind", ["few", "many"])
def test_the_model_sees_a_last_commit_that_nobody_waits_for(kind):
    with pytest.raises(AssertionError, match="still under way"):
        for seed in range(300):
            run, _ = _make(kind, seed, 5)
            run.drains = False
            run.run()


@pytest.mark.parametrize("mistake", ["scales too few", "S not let go of", "P before O", "one barrier for both halves"])
def test_the_model_sees_a_mistake(mistake):
    """Each way of getting out of step that the protocols avoid is seen when it is put into the model."""
    with pytest.raises(AssertionError):
        for seed in range(300):
            run, _ = _make("many" if mistake in ("scales too few", "one barrier for both halves") else "few", seed, 20)
            if mistake == "scales too few":
                run.scales -= 3
            elif mistake == "S not let go of":
                run.s_free.over = lambda phase: True
            elif mistake == "P before O":
                run.o_full.over = lambda phase: True
            else:
                for d in range(2):
                    run.o_step[d][1] = run.o_step[d][0]
            run.run()
