"""The barriers of paged_attention_kernel, modelled on the CPU.

Every role of the kernel (csrc/kvd_paged_attn.cuh) is a generator that yields the barrier phase it waits for; copies and the commits of MMAs
are events that come later (those of one warp in their order).  The roles run in random order.  A parity tells a phase only from its
neighbours, so a wait is also checked against the phase that is meant: a barrier that ran two phases ahead of a waiting warp, or that a warp
waits on two phases early, is a fault, as is a ring stage that holds another tile than its reader expects, and a deadlock.
"""

import random

import pytest

JOBS = 4  # records of the job ring


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.done = name, count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.count

    def over(self, phase):
        """Whether a wait for this phase's parity returns; it has to say what the phase itself says."""
        says = (self.done - 1) & 1 == phase & 1
        assert says == (self.done > phase), "%s: %d phases done, a wait for phase %d says %s" % (self.name, self.done, phase, says)
        return says


def k_place(job, t):
    return 2 * t if job["dual"] else t if t < 2 else 2 * t - 1


def v_place(job, t):
    return 2 * t + 1 if job["dual"] else min(2 * t + 2, 2 * job["n"] - 1)


class Model:
    def __init__(self, jobs, stages, rng):
        self.jobs, self.stages, self.rng = jobs, stages, rng
        bars = lambda name, n, count: [Bar(name + str(i), count) for i in range(n)]  # noqa: E731
        self.job_full, self.job_empty = bars("job_full", JOBS, 1), bars("job_empty", JOBS, 7)
        self.q_full, self.q_empty = Bar("q_full", 1), Bar("q_empty", 2)
        self.kv_full, self.kv_empty = bars("kv_full", stages, 1), bars("kv_empty", stages, 2)
        self.s_full, self.p_ready, self.o_full, self.o_empty, self.ml_full, self.tail_go, self.tail_ready, self.pace = (
            bars(n, 2, 1) for n in ("s_full", "p_ready", "o_full", "o_empty", "ml_full", "tail_go", "tail_ready", "pace"))
        self.slot, self.holds, self.cleared = [None] * JOBS, {}, set()
        self.later = {"K": [], "V": [], "Q": [], "MMA0": [], "MMA1": []}

    # ---- roles

    def scheduler(self):
        for i, job in enumerate(self.jobs + [{"n": 0}]):
            if i >= JOBS:
                yield self.job_empty[i % JOBS], i // JOBS - 1
            self.slot[i % JOBS] = job
            self.job_full[i % JOBS].arrive()

    def each_job(self, late=False):
        """Yields waits, then ("job", record); the record is let go of at once, or (late) when the caller asks for the next."""
        i = 0
        while True:
            yield self.job_full[i % JOBS], i // JOBS
            job = self.slot[i % JOBS]
            if job["n"] == 0:
                return
            if not late:
                self.job_empty[i % JOBS].arrive()
            yield "job", job
            if late:
                self.job_empty[i % JOBS].arrive()
            i += 1

    def over_jobs(self, body, late=False):
        for step in self.each_job(late):
            if step[0] == "job":
                yield from body(step[1])
            else:
                yield step

    def loader(self, is_v):
        ring, items = 0, 0

        def body(job):
            nonlocal ring, items
            for t in range(job["n"]):
                at = ring + (v_place(job, t) if is_v else k_place(job, t))
                stage, turn = at % self.stages, at // self.stages
                if turn > 0:
                    yield self.kv_empty[stage], turn - 1

                def land(stage=stage, at=at):
                    self.holds[stage] = at
                    self.kv_full[stage].arrive()

                self.later["V" if is_v else "K"].append(land)
                yield None
                if t == 0 and not is_v:
                    if items > 0:
                        yield self.q_empty, items - 1
                    self.later["Q"].append(self.q_full.arrive)
                    items += 1
            ring += 2 * job["n"]

        return self.over_jobs(body)

    def mma(self, d):
        ring, items, uses, tails, p_phase, pairs = 0, 0, 0, 0, 0, 0
        commit = self.later["MMA%d" % d].append

        def body(job):
            nonlocal ring, items, uses, tails, p_phase, pairs
            n, dual, at = job["n"], job["dual"], ring
            yield self.q_full, items
            step = 1 if dual else 2

            def stage_there():
                return self.kv_full[at % self.stages], at // self.stages

            def take():
                nonlocal at
                assert self.holds[at % self.stages] == at, "a stage holds tile %d, not %d" % (self.holds[at % self.stages], at)
                at += 1
                return (at - 1) % self.stages

            for j in range(-step, n):
                more = j + step < n
                if not dual and j & 1 != d:
                    for there in (j >= 0, more):
                        if there:
                            yield stage_there()
                            commit(self.kv_empty[take()].arrive)
                            yield None
                    continue
                v = None
                if j >= 0:
                    yield stage_there()
                    if j == job["tail"] and (not dual or d == 0):
                        self.tail_go[d].arrive()
                        yield self.tail_ready[d], tails
                        tails += 1
                    v = take()
                    if j < step and uses > 0:
                        yield self.o_empty[d], uses - 1
                    yield self.p_ready[d], p_phase
                    p_phase += 1
                    if dual and (d == 1 or pairs > 0):
                        yield self.pace[d ^ 1], pairs - (d ^ 1)
                    assert j != job["tail"] or ring + v_place(job, j) in self.cleared, "P V with an end that was not cleared"
                    if not more:
                        commit(self.o_full[d].arrive)
                if more:
                    yield stage_there()
                    k = take()
                    commit(self.s_full[d].arrive)
                    commit(self.kv_empty[k].arrive)
                    if j + 2 * step >= n:
                        commit(self.q_empty.arrive)
                if j >= 0:
                    commit(self.kv_empty[v].arrive)
                    if dual:
                        self.pace[d].arrive()
                        pairs += 1
                yield None
            if not dual and n == 1 and d == 1:
                self.q_empty.arrive()
            else:
                uses += 1
            ring, items = ring + 2 * n, items + 1

        return self.over_jobs(body)

    def ends_of_v(self):
        ring, went = 0, [0, 0]

        def body(job):
            nonlocal ring
            t = job["tail"]
            if t >= 0:
                s = 0 if job["dual"] else t & 1
                yield self.tail_go[s], went[s]
                went[s] += 1
                at = ring + v_place(job, t)
                assert self.holds[at % self.stages] == at
                yield None
                assert self.holds[at % self.stages] == at
                self.cleared.add(at)
                self.tail_ready[s].arrive()
            ring += 2 * job["n"]

        return self.over_jobs(body)

    def softmax(self, d):
        s_phase, o_phase, joins = 0, [0, 0], 0

        def body(job):
            nonlocal s_phase, joins
            dual, two = job["dual"], not job["dual"] and job["n"] > 1
            for _ in range(job["n"] if dual else (job["n"] - d + 1) // 2):
                yield self.s_full[d], s_phase
                s_phase += 1
                yield None
                self.p_ready[d].arrive()
            if two:
                if d == 1:
                    self.ml_full[joins & 1].arrive()
                else:
                    yield self.ml_full[joins & 1], joins >> 1
                joins += 1
            if dual or d == 0:
                yield self.o_full[d], o_phase[d]
                if two:
                    yield self.o_full[1], o_phase[1]
                yield None
                if two:
                    self.o_empty[1].arrive()
                self.o_empty[d].arrive()
            o_phase[0] += 1
            o_phase[1] += 1 if dual or two else 0

        return self.over_jobs(body, late=True)

    # ---- the run

    def run(self):
        roles = {"scheduler": self.scheduler(), "K": self.loader(False), "V": self.loader(True), "MMA0": self.mma(0), "MMA1": self.mma(1),
                 "ends": self.ends_of_v(), "soft0": self.softmax(0), "soft1": self.softmax(1)}
        waits = dict.fromkeys(roles)
        speed = {k: self.rng.choice([1, 1, 5, 20]) for k in list(roles) + ["later " + k for k in self.later]}
        while roles:
            able = [k for k in roles if waits[k] is None or waits[k][0].over(waits[k][1])]
            able += ["later " + k for k, events in self.later.items() if events]
            assert able, "deadlock: %s" % {k: (waits[k][0].name, waits[k][0].done, waits[k][1]) for k in roles}
            k = self.rng.choices(able, [speed[a] for a in able])[0]
            if k.startswith("later "):
                events = self.later[k[6:]]
                events.pop(0 if k[6:].startswith("MMA") else self.rng.randrange(len(events)))()
                continue
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k]


@pytest.mark.parametrize("stages", [5, 10])  # head size 128 and 64
@pytest.mark.parametrize("duals", [0.0, 0.05, 0.4, 0.9])
def test_roles_keep_in_step(stages, duals):
    for seed in range(150):
        rng = random.Random(1000 * stages + 10 * seed + int(9 * duals))
        jobs = []
        for _ in range(rng.randint(1, 25)):
            n = rng.choice([1, 1, 1, 2, 2, 3, 4, 5, 6, 9])
            jobs.append({"n": n, "dual": rng.random() < duals, "tail": rng.choice([-1, n - 1, n - 1, rng.randrange(n)])})
        Model(jobs, stages, rng).run()


@pytest.mark.parametrize("mistake", ["let go of at once", "told for every item", "no turns"])
def test_the_model_sees_a_mistake(mistake):
    """Each way of getting out of step that the protocol avoids is seen when it is put into the model."""

    class Wrong(Model):
        def mma(self, d):
            if mistake == "no turns":
                self.pace[0].over = self.pace[1].over = lambda phase: True
            if mistake == "let go of at once":
                commits, empty = self.later["MMA%d" % d], {id(b) for b in self.kv_empty}

                class Eager(list):
                    def append(self, event):
                        if not commits or id(event.__self__) not in empty:
                            list.append(self, event)
                        else:
                            event()

                self.later["MMA%d" % d] = commits = Eager()
            return super().mma(d)

        def softmax(self, d):
            for step in super().softmax(d):
                yield step
                if mistake == "told for every item" and d == 0 and step is not None and step[0] is self.o_full[0]:
                    self.o_empty[1].arrive()

    with pytest.raises(AssertionError):
        for seed in range(200):
            rng = random.Random(seed)
            jobs = []
            for _ in range(20):
                n = rng.choice([1, 1, 2, 3, 4, 5])
                jobs.append({"n": n, "dual": rng.random() < 0.4, "tail": rng.choice([-1, n - 1, rng.randrange(n)])})
            Wrong(jobs, 5, rng).run()


class Abandoned(Model):
    """A run that is given up: every role goes on until it has to wait and leaves there, and then, with all of them at the kernel's end, the
    copies and MMAs still under way are waited for.  mistake: what that end forgets."""

    mistake = None

    def __init__(self, *args):
        super().__init__(*args)
        self.kv_loads, self.q_loads, self.left_early = [0] * self.stages, 0, set()

    def loader(self, is_v):
        role = super().loader(is_v)
        list_of, q_of = self.later["V" if is_v else "K"], self.later["Q"]
        seen, seen_q = 0, 0

        class Counted(list):  # what the loading warps note as they ask for a copy
            def append(inner, event):
                stage, at = event.__defaults__
                self.kv_loads[stage] = at // self.stages + 1
                list.append(inner, event)

        class CountedQ(list):
            def append(inner, event):
                self.q_loads += 1
                list.append(inner, event)

        if not isinstance(list_of, Counted):
            self.later["V" if is_v else "K"] = Counted(list_of)
        if not is_v and not isinstance(q_of, CountedQ):
            self.later["Q"] = CountedQ(q_of)
        return role

    def happen(self, name):
        events = self.later[name]
        events.pop(0 if name.startswith("MMA") else self.rng.randrange(len(events)))()

    def run(self, moves):
        roles = {"scheduler": self.scheduler(), "K": self.loader(False), "V": self.loader(True), "MMA0": self.mma(0), "MMA1": self.mma(1),
                 "ends": self.ends_of_v(), "soft0": self.softmax(0), "soft1": self.softmax(1)}
        waits = dict.fromkeys(roles)

        def move(k):
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k]

        able = lambda: [k for k in roles if waits[k] is None or waits[k][0].over(waits[k][1])]  # noqa: E731
        for _ in range(moves):
            choice = able() + ["later " + k for k, events in self.later.items() if events]
            if not choice:
                break
            k = self.rng.choice(choice)
            self.happen(k[6:]) if k.startswith("later ") else move(k)
        self.left_early = {"K", "V"} - set(roles)
        while True:  # given up
            k = self.rng.choice(able() or [None])
            if k is None:
                break
            move(k)

        def wait_for(bar, phases, names):
            while bar.done < phases:
                names = [n for n in names if self.later[n]]
                assert names, "the end waits for a copy that nobody asked for"
                self.happen(self.rng.choice(names))

        wait_for_mmas = [n for n in ("MMA0", "MMA1") if self.mistake != "mmas"]
        for n in wait_for_mmas:
            while self.later[n]:
                self.happen(n)
        if not (self.mistake == "loads done" and self.left_early):
            for stage, n in enumerate(self.kv_loads):
                wait_for(self.kv_full[stage], n, ["K", "V"])
        if self.mistake != "q":
            wait_for(self.q_full, self.q_loads, ["Q"])
        assert not any(self.later.values()), "still under way at the end: %s" % {k: len(v) for k, v in self.later.items() if v}


def _drawn_jobs(rng, most):
    jobs = []
    for _ in range(rng.randint(1, most)):
        n = rng.choice([1, 1, 2, 3, 4, 5, 9])
        jobs.append({"n": n, "dual": rng.random() < 0.4, "tail": rng.choice([-1, n - 1, rng.randrange(n)])})
    return jobs


@pytest.mark.parametrize("stages", [5, 10])
def test_nothing_is_under_way_when_a_run_is_given_up(stages):
    for seed in range(600):
        rng = random.Random(seed)
        Abandoned(_drawn_jobs(rng, 12), stages, rng).run(int(2 ** rng.uniform(0, 10)))


@pytest.mark.parametrize("mistake", ["q", "mmas", "loads done"])
def test_the_model_sees_what_an_end_forgets(mistake):
    """Q's copy; MMAs; the copies of a loading warp that was through when the run was given up."""
    with pytest.raises(AssertionError, match="still under way"):
        for seed in range(600):
            rng = random.Random(seed)
            run = Abandoned(_drawn_jobs(rng, 3), 10, rng)
            run.mistake = mistake
            run.run(int(2 ** rng.uniform(0, 10)))


class Pieces:
    """The joins of a small call: CTAs whose four warps each write their rows of a piece, one of which takes a ticket for it; the holder of an
    item's last ticket has its warps join.  Some CTAs are given up at some moment and take the tickets they owe on their way out."""

    owes = True

    def __init__(self, items, rng):
        # items: the CTAs that hold each one's pieces, in order; a CTA ends its items in that order
        self.items, self.rng, self.words = items, rng, {}

    def launch(self, nonce, give_up):
        rng, items, words = self.rng, self.items, self.words
        ctas = sorted({c for held in items for c in held})
        written, joined, gone, open_ = set(), [], set(), {}

        def ticket(i):
            old, count = words.get(i, (None, 0))
            count = count + 1 if old == nonce else 1
            words[i] = (nonce, count) if count < len(items[i]) else (0, 0)
            return count == len(items[i])

        def cta(c):
            """Yields (warp, condition) until the CTA is done: a scheduler of its own over its four warps."""
            mine = [i for i, held in enumerate(items) if c in held]
            piece_done, verdict, joins, taken = Bar("piece_done", 4), Bar("verdict", 1), {}, 0

            def warp(w):
                nonlocal taken
                for cuts, i in enumerate(mine):
                    yield None
                    written.add((i, c, w))
                    piece_done.arrive()
                    if w == 0:
                        yield piece_done, cuts
                        joins[cuts] = ticket(i)
                        taken += 1
                        verdict.arrive()
                    yield verdict, cuts
                    if joins[cuts]:
                        if not gone:
                            assert {(i, x, y) for x in items[i] for y in range(4)} <= written, "joined before every piece was there"
                        joined.append((i, w))

            warps, waits = {w: warp(w) for w in range(4)}, dict.fromkeys(range(4))
            left = rng.randrange(12) if c in give_up else 1 << 30
            while warps:
                able = [w for w in warps if waits[w] is None or waits[w][0].over(waits[w][1])]
                if left <= 0:  # given up: whoever has to wait leaves
                    able = [w for w in able if waits[w] is not None or rng.random() < 0.5]
                    if not able:
                        gone.add(c)
                        break
                w = rng.choice(able)
                left -= 1
                try:
                    waits[w] = next(warps[w])
                except StopIteration:
                    del warps[w]
                yield
            if c in gone and self.owes:
                for i in mine[taken:]:
                    yield
                    ticket(i)

        open_ = {c: cta(c) for c in ctas}
        while open_:
            c = rng.choice(list(open_))
            try:
                next(open_[c])
            except StopIteration:
                del open_[c]
        if not gone:
            assert sorted(joined) == [(i, w) for i in range(len(items)) for w in range(4)], "an item joined twice or not at all"
        return bool(gone)


def _drawn_items(rng):
    """Items cut over neighbouring CTAs: each begins where the last one ended."""
    items, c = [], 0
    for _ in range(rng.randint(1, 5)):
        n = rng.randint(2, 5)
        items.append(list(range(c, c + n)))
        c += n - (rng.random() < 0.6)
    return items


def test_pieces_are_joined_once_and_after_launches_given_up():
    """Replays of a graph (one nonce) and other calls on one workspace, some of them given up: the next one joins every item once."""
    given_up = 0
    for seed in range(400):
        rng = random.Random(seed)
        run = Pieces(_drawn_items(rng), rng)
        run.words = {i: rng.choice([(None, 0), (7, 3), (8, 1)]) for i in range(len(run.items))}  # what the memory held
        ctas = sorted({c for held in run.items for c in held})
        for _ in range(5):
            nonce = rng.choice([1, 1, 2])
            give_up = set(rng.sample(ctas, rng.randint(1, 2))) if rng.random() < 0.5 else set()
            given_up += run.launch(nonce, give_up)
            assert all(count == 0 for _, count in run.words.values())
    assert given_up > 100


def test_the_model_sees_tickets_that_are_owed():
    class Wrong(Pieces):
        owes = False

    with pytest.raises(AssertionError, match="joined"):
        for seed in range(400):
            rng = random.Random(seed)
            run = Wrong(_drawn_items(rng), rng)
            ctas = sorted({c for held in run.items for c in held})
            for give_up in ({rng.choice(ctas)}, set(), set()):
                run.launch(1, give_up)
