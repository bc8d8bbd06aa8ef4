"""A model of the prompt kernel's barriers (csrc/prompt.cuh): who waits for which phase of which barrier, and who arrives there.

A barrier tells its phases apart by parity alone: a wait for phase x ends when x + 1 phases are complete, but also when x - 1 are
(too early), and not when x + 2 are (never, maybe). `run` plays the roles in a random order, some of them held back for a while, and
raises `Lost` where a wait meets a barrier that is not at its phase or the next one, or where nobody can go on."""
import random

META = 8


class Lost(Exception):
    pass


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.phases = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phases = self.count, self.phases + 1


class Kernel:
    """wide: heads of more than 128 values; fp8: codes through stages; boxes: TMA boxes, or rows one by one; q_box: queries as boxes.
    Warps that do the same (four softmax warps of a tile, helpers) are two each, which can run apart."""

    def __init__(self, segments, wide, fp8, boxes, q_box, rng, loader_fills=True, second_waits="final"):
        self.segments, self.wide, self.fp8, self.boxes, self.q_box, self.rng = segments, wide, fp8, boxes, q_box, rng
        self.loader_fills, self.second_waits = loader_fills, second_waits
        self.slots, self.stages, self.parts = (3 if fp8 else 4), 3, (2 if wide else 1)
        self.loaders = 2 if boxes else 1
        self.helpers = 4 if fp8 and boxes else 2
        fills = self.helpers + (1 if loader_fills else 0) if not boxes else self.helpers // 2 if fp8 else self.loaders
        bars = lambda name, n, count: [Barrier(f"{name}[{i}]", count) for i in range(n)]  # noqa: E731
        self.full, self.empty = bars("full", self.slots, fills), bars("empty", self.slots, 1)
        self.st_full, self.st_empty = bars("st_full", self.stages, self.loaders), bars("st_empty", self.stages, self.helpers)
        self.q_full, self.q_empty = Barrier("q_full", 1 if q_box else self.helpers), Barrier("q_empty", 1)
        self.k_meta, self.v_go, self.v_meta = bars("k_meta", META, 1), bars("v_go", META, 1), bars("v_meta", META, self.helpers)
        self.s_full, self.p_full = bars("s_full", 2, 1), bars("p_full", 2, 2)
        self.o_final, self.o_done = [bars("o_final", 2, 1) for _ in range(2)], Barrier("o_done", 1)
        self.seg_full, self.seg_empty = bars("seg_full", 2, 1), bars("seg_empty", 2, 4 + 1 + self.loaders + self.helpers)
        self.commits, self.landing = [], []

    # ---- what a role does: (barrier, phase) is waited for, None lets others go on
    def each_segment(self, end):
        for k, s in enumerate(self.segments):
            yield self.seg_full[k & 1], k >> 1
            yield from end(k, s)
        yield self.seg_full[len(self.segments) & 1], len(self.segments) >> 1

    def hand_out(self):
        for k in range(len(self.segments) + 1):
            if k >= 2:
                yield self.seg_empty[k & 1], (k >> 1) - 1
            self.seg_full[k & 1].arrive()
            yield None

    def order(self, T, lead):
        """Key and value tiles as they are brought in: (whether values, tile)."""
        k = v = 0
        while v < T:
            values = k == min(T, v + lead)
            yield values, (v if values else k)
            v, k = v + values, k + (not values)

    def lead(self, s):
        return 1 if not self.wide and s["nt"] == 2 else 2

    def load(self, loader):
        st = dict(slot=0, kn=0, pc=0)

        def segment(k, s):
            for values, n in self.order(s["T"], self.lead(s)):
                if not values and loader == 0:
                    yield None                        # pages are looked up
                    self.k_meta[(st["kn"] + n) % META].arrive()
                for part in range(self.parts):
                    at = st["slot"]
                    st["slot"] += 1
                    ring, ready = (self.st_empty, self.st_full) if self.fp8 and self.boxes else (self.empty, self.full)
                    yield ring[at % len(ring)], at // len(ring) - 1
                    if values and part + 1 == self.parts and loader == 0 and s["partly"][n]:
                        self.v_go[st["pc"] % META].arrive()
                        st["pc"] += 1
                    if self.boxes:
                        self.landing.append(ready[at % len(ring)])
                    elif self.loader_fills:
                        ready[at % len(ring)].arrive()
            st["kn"] += s["T"]
            self.seg_empty[k & 1].arrive()
        yield from self.each_segment(segment)

    def help(self, w):
        st = dict(pc=0, seq=0)

        def segment(k, s):
            T = s["T"]
            if (not self.q_box or w == 0) and k > 0:
                yield self.q_empty, k - 1
            if self.q_box and w == 0:
                self.landing.append(self.q_full)
            elif not self.q_box:
                yield None
                self.q_full.arrive()

            def note():
                self.v_meta[st["pc"] % META].arrive()
                st["pc"] += 1
            if self.boxes and not self.fp8:
                for n in range(T):
                    if s["partly"][n]:
                        yield self.v_go[st["pc"] % META], st["pc"] // META
                        for part in range(self.parts):
                            at = st["seq"] + (min(T, n + self.lead(s)) + n) * self.parts + part
                            yield self.full[at % self.slots], at // self.slots
                        note()
                st["seq"] += 2 * T * self.parts
            else:
                for values, n in self.order(T, self.lead(s)):
                    for part in range(self.parts):
                        at = st["seq"]
                        st["seq"] += 1
                        if self.boxes:
                            yield self.st_full[at % self.stages], at // self.stages
                            if (at & 1) != w // 2:
                                self.st_empty[at % self.stages].arrive()
                                continue
                        if at >= self.slots:
                            yield self.empty[at % self.slots], at // self.slots - 1
                        yield None
                        if self.boxes:
                            self.st_empty[at % self.stages].arrive()
                            yield None
                        self.full[at % self.slots].arrive()
                    if values and s["partly"][n]:
                        note()
            self.seg_empty[k & 1].arrive()
        yield from self.each_segment(segment)

    def multiply(self):
        st = dict(slot=0, pc=0, used=[0, 0])

        def next_full():
            at = st["slot"]
            st["slot"] += 1
            return self.full[at % self.slots], at // self.slots, self.empty[at % self.slots]

        def looked_through(s, n):
            if s["partly"][n]:
                yield self.v_meta[st["pc"] % META], st["pc"] // META
                st["pc"] += 1

        def segment(k, s):
            T, commit = s["T"], self.commits.append
            yield self.q_full, k
            if not self.wide and s["nt"] == 2:
                f, x, e = next_full()
                yield f, x
                for t in range(2):
                    commit(self.s_full[t])
                commit(e)
                if T == 1:
                    commit(self.q_empty)
                for n in range(T):
                    f, x, ve = next_full()
                    yield f, x
                    yield from looked_through(s, n)
                    for t in range(2):
                        yield self.p_full[t], st["used"][t] + n
                        if t == 1:
                            commit(ve)
                        if n + 1 < T:
                            if t == 0:
                                f, x, ke = next_full()
                                yield f, x
                            commit(self.s_full[t])
                        else:
                            commit(self.o_final[t][k & 1])
                    if n + 1 < T:
                        commit(ke)
                        if n + 2 == T:
                            commit(self.q_empty)
                st["used"] = [u + T for u in st["used"]]
            else:
                def keys(n):
                    for _ in range(self.parts):
                        f, x, e = next_full()
                        yield f, x
                        commit(e)
                    commit(self.s_full[n & 1])
                    if n + 1 == T:
                        commit(self.q_empty)
                yield from keys(0)
                if T > 1:
                    yield from keys(1)
                for n in range(T):
                    yield self.p_full[n & 1], st["used"][n & 1] + (n >> 1)
                    yield from looked_through(s, n)
                    for _ in range(self.parts):
                        f, x, e = next_full()
                        yield f, x
                        commit(e)
                    commit(self.o_done)
                    if n + 1 == T:
                        commit(self.o_final[0][k & 1])
                        if not self.wide:
                            commit(self.o_final[1][k & 1])
                    if n + 2 < T:
                        yield from keys(n + 2)
                st["used"] = [st["used"][0] + (T + 1) // 2, st["used"][1] + T // 2]
            yield None
            self.seg_empty[k & 1].arrive()
        yield from self.each_segment(segment)

    def softmax(self, tile):
        st = dict(used=[0, 0], kn=0, pc=0, dones=0)

        def segment(k, s):
            T, nt = s["T"], s["nt"]
            if tile < nt and not (self.wide and tile):
                count = [st["used"][tile if nt == 2 else 0], st["used"][1]]
                for n in range(T):
                    buf = tile if nt == 2 else n & 1
                    at = st["kn"] + n
                    yield self.k_meta[at % META], at // META
                    which = 0 if nt == 2 or buf == 0 else 1
                    yield self.s_full[buf], count[which]
                    count[which] += 1
                    if nt == 1 and n > 0 and self.rng.random() < 0.2:
                        yield self.o_done, st["dones"] + n - 1
                    if s["partly"][n]:
                        yield self.v_meta[st["pc"] % META], st["pc"] // META
                        st["pc"] += 1
                    yield None
                    self.p_full[buf].arrive()
                yield self.o_final[tile][k & 1], k >> 1
                for _ in range(self.rng.choice([0, 0, 3, 60])):   # outputs, a join
                    yield None
            elif not self.wide:
                if self.second_waits == "scores":
                    for n in range(1, T, 2):
                        yield self.s_full[1], st["used"][1] + (n >> 1)
                else:
                    yield self.o_final[1][k & 1], k >> 1
                st["pc"] += sum(s["partly"])
            if nt == 2:
                st["used"] = [u + T for u in st["used"]]
            else:
                st["used"] = [st["used"][0] + (T + 1) // 2, st["used"][1] + T // 2]
                st["dones"] += T
            st["kn"] += T
            self.seg_empty[k & 1].arrive()
        yield from self.each_segment(segment)

    def tensor_cores(self):                           # commits arrive in the order in which they were made
        while True:
            if self.commits:
                self.commits.pop(0).arrive()
                yield None
            else:
                yield "idle"

    def memory(self):                                 # boxes land in any order
        while True:
            if self.landing:
                self.landing.pop(self.rng.randrange(len(self.landing))).arrive()
                yield None
            else:
                yield "idle"


def run(segments, wide, fp8, boxes, q_box, seed, **how):
    rng = random.Random(seed)
    k = Kernel(segments, wide, fp8, boxes, q_box, rng, **how)
    roles = {"hand out": k.hand_out(), "multiply": k.multiply()}
    roles |= {f"load {i}": k.load(i) for i in range(k.loaders)} | {f"help {i}": k.help(i) for i in range(k.helpers)}
    roles |= {f"softmax {t}.{i}": k.softmax(t) for t in range(2) for i in range(2)}
    engines = {"tensor cores": k.tensor_cores(), "memory": k.memory()}
    waits = {name: None for name in roles}
    held, until, step = set(), 0, 0
    while waits:
        step += 1
        if step >= until:                             # some are held back for a while
            names = [*waits, *engines]
            held = set(rng.sample(names, rng.choice([0, 1, 1, 2, len(names) // 2])))
            until = step + rng.choice([5, 30, 200])
        ready = [n for n in (*waits, *engines) if n not in held]
        rng.shuffle(ready)
        for name in ready:
            if name in engines:
                if next(engines[name]) == "idle":
                    continue
                break
            if waits[name] is not None:
                bar, x = waits[name]
                if not x <= bar.phases <= x + 1:
                    raise Lost(f"{name} waits for phase {x} of {bar.name}, which has had {bar.phases}")
                if bar.phases != x + 1:
                    continue
            try:
                waits[name] = next(roles[name])
            except StopIteration:
                del waits[name]
            break
        else:
            if not held:
                raise Lost("nobody can go on: " + ", ".join(f"{n}: {w and (w[0].name, w[1])}" for n, w in waits.items()))
            until = step


def segments_of(rng, wide):
    n = rng.choice([1, 1, 2, 3, 6])
    return [dict(T=(T := rng.choice([1, 1, 2, 3, 4, 9])), nt=1 if wide else rng.choice([1, 2]), partly=[rng.random() < rng.choice([0.1, 0.9]) for _ in range(T)])
            for _ in range(n)]
