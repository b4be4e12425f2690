"""Randomised-schedule model of the tensor-core scan's pipeline (CPU, no GPU).

A block of the kernel (csrc/scan_tc.cu) walks units of some chunks each (none, for an empty
sequence): a planner hands them to every role through a ring of two, a TMA warp loads q, k and v,
two warps issue the products, and the warps of rows, tokens and state columns do the rest. The
roles meet at mbarriers, whose waits test a phase by its parity. Here each role is a coroutine
(two for each group of warps, which need not run together), loads and products end when chance
has it (products of one warp in order), and every schedule is checked: each wait passes for its
own phase, each reader sees the chunk it is at for as long as it reads, nothing is overwritten
early, and no schedule stops. With the order that the TMA warp must not take (the next unit
first, the last chunk's q after it) the model stops where units without chunks follow one another."""

import random

import pytest

SLOTS = 5  # chunks whose decays are held


class MBarrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.done = self.tx = 0

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        self.settle()

    def landed(self, tx):
        self.tx -= tx
        self.settle()

    def settle(self):
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count


class Stopped(Exception):
    pass


class Block:
    def __init__(self, units, local, seed, q_first=True):
        self.units, self.local, self.q_first = units, local, q_first
        self.rnd = random.Random(seed)
        self.nu = 2 if local else 1  # buffers of U and of dS
        b = self.bar = {}
        for name, count in dict(q_full=1, q_empty=1, c_full=1, p_full=2, y_full=1, y_free=2, s_full=2).items():
            b[name] = MBarrier(count)
        for i in range(2):
            b["k_full", i], b["k_empty", i] = MBarrier(1), MBarrier(1 if local else 2)
            b["v_full", i], b["v_empty", i] = MBarrier(1), MBarrier(2 if local else 1)
            b["u_full", i], b["ds_full", i], b["ds_free", i] = MBarrier(2), MBarrier(1), MBarrier(2)
            b["unit_full", i], b["unit_empty", i] = MBarrier(1), MBarrier(6 if local else 9)
        for i in range(SLOTS):
            b["da_full", i] = MBarrier(1)
        self.holds = {}            # what each buffer holds: the number of a chunk
        self.loads, self.queues = [], {"Q": [], "U": []}
        self.ring = [None, None]
        self.ends = [0, 0]         # final states stored, by half

    # ------------------------------------------------------------------ what roles do
    def wait(self, name, phase):
        bar = self.bar[name]
        while (bar.done & 1) == (phase & 1):
            yield name
        assert bar.done == phase + 1, f"{name}: a wait for phase {phase} passed at {bar.done}"
        yield None

    def see(self, n, *buffers):
        for x in buffers:
            assert self.holds.get(x) == n, f"{x} holds {self.holds.get(x)}, wanted {n}"

    def take(self, k):
        yield from self.wait(("unit_full", k & 1), k >> 1)
        number, chunks = self.ring[k & 1]
        assert number == k
        self.bar["unit_empty", k & 1].arrive()
        return chunks

    def load(self, buffer, n, name):
        self.bar[name].arrive(tx=1)
        self.loads.append((buffer, n, name))

    def product(self, warp, n, reads, writes):
        self.queues[warp].append(["product", n, reads, writes, False])

    def commit(self, warp, name):
        self.queues[warp].append(["commit", name])

    # ------------------------------------------------------------------ the roles
    def plan(self):
        for k, chunks in enumerate(self.units + [-1]):
            if k >= 2:
                yield from self.wait(("unit_empty", k & 1), (k >> 1) - 1)
            self.ring[k & 1] = (k, chunks)
            self.bar["unit_full", k & 1].arrive()
            yield None

    def tma(self):
        n = k = c = chunks = nq = 0
        due = False  # a chunk whose q is still to be loaded

        def load_q(nq):
            if nq >= 1:
                yield from self.wait("q_empty", nq - 1)
            self.load("q", nq, "q_full")

        while chunks >= 0:
            if self.q_first and due and not self.local:
                yield from load_q(nq)
                nq += 1
            while 0 <= chunks <= c:
                chunks = yield from self.take(k)
                k, c = k + 1, 0
            if not self.q_first and due and not self.local:
                yield from load_q(nq)
                nq += 1
            if chunks < 0:
                break
            b = n & 1
            if n >= 2:
                yield from self.wait(("k_empty", b), (n >> 1) - 1)
            self.load(("k", b), n, ("k_full", b))
            if n >= 2:
                yield from self.wait(("v_empty", b), (n >> 1) - 1)
            self.load(("v", b), n, ("v_full", b))
            n, c, due = n + 1, c + 1, True

    def over_chunks(self, body, start=None, end=None):
        n = k = 0
        while (chunks := (yield from self.take(k))) >= 0:
            if start:
                start(n, chunks)
            for c in range(chunks):
                yield from body(n, c, chunks)
                n += 1
            if end:
                end()
            k += 1

    def mma_q(self):
        def body(n, c, chunks):
            b = n & 1
            yield from self.wait("q_full", n)
            yield from self.wait(("k_full", b), n >> 1)
            if n >= 1:
                yield from self.wait("y_full", n - 1)
            self.product("Q", n, ["q", ("k", b)], ["C"])
            self.commit("Q", "c_full")
            yield from self.wait("s_full", n)
            if n >= 1:
                yield from self.wait("y_free", n - 1)
            self.product("Q", n, ["q", ("S", 0), ("S", 1)], ["Y2"])
            self.commit("Q", "q_empty")
            self.commit("Q", ("k_empty", b))

        return self.over_chunks(body)

    def mma_u(self):
        def body(n, c, chunks):
            b, u = n & 1, n % self.nu
            yield from self.wait(("u_full", u), n // self.nu)
            yield from self.wait(("k_full", b), n >> 1)
            if n >= self.nu:
                yield from self.wait(("ds_free", u), n // self.nu - 1)
            if not self.local:
                yield from self.wait("c_full", n)
            self.product("U", n, [("k", b), ("U", u, 0), ("U", u, 1)], [("dS", u)])
            self.commit("U", ("ds_full", u))
            self.commit("U", ("k_empty", b))
            if self.local:
                return
            yield from self.wait("p_full", n)
            yield from self.wait(("v_full", b), n >> 1)
            self.product("U", n, [("P", 0), ("P", 1), ("v", b)], ["Y1"])
            self.commit("U", "y_full")
            self.commit("U", ("v_empty", b))

        return self.over_chunks(body)

    def rows(self, half):
        def body(n, c, chunks):
            decays = ("decays", n % SLOTS)
            yield from self.wait(("da_full", n % SLOTS), n // SLOTS)
            yield from self.wait("c_full", n)
            self.see(n, decays, "C")
            yield None
            self.holds["P", half] = n  # over its part of C
            self.bar["p_full"].arrive()
            yield from self.wait("y_full", n)
            yield from self.wait("q_empty", n)
            self.see(n, decays, "Y1", "Y2")
            yield None
            self.see(n, decays, "Y1", "Y2")
            self.bar["y_free"].arrive()

        return self.over_chunks(body)

    def tokens(self, half):
        def body(n, c, chunks):
            b, u, slot = n & 1, n % self.nu, n % SLOTS
            if half == 0:
                self.holds["decays", slot] = n
                self.bar["da_full", slot].arrive()
                yield None
            yield from self.wait(("da_full", slot), n // SLOTS)
            self.see(n, ("decays", slot))
            yield from self.wait(("v_full", b), n >> 1)
            if n >= self.nu:
                yield from self.wait(("ds_full", u), n // self.nu - 1)
            if c + 1 == chunks:  # tokens behind the sequence become zeros in k
                yield from self.wait(("k_full", b), n >> 1)
                self.see(n, ("k", b))
            self.see(n, ("v", b))
            self.holds["U", u, half] = n
            yield None
            self.see(n, ("v", b))
            self.bar["u_full", u].arrive()
            if self.local:
                self.bar["v_empty", b].arrive()

        return self.over_chunks(body)

    def state(self, half):
        def start(n, chunks):
            if not self.local and chunks > 0:
                self.holds["S", half] = n
                self.bar["s_full"].arrive()

        def end():
            self.ends[half] += 1

        def body(n, c, chunks):
            u = n % self.nu
            yield from self.wait(("ds_full", u), n // self.nu)
            if not self.local:
                yield from self.wait("q_empty", n)
            self.see(n, ("dS", u), ("decays", n % SLOTS))
            yield None
            self.see(n, ("dS", u), ("decays", n % SLOTS))
            put = not self.local and c + 1 < chunks
            if put:
                self.holds["S", half] = n + 1
            self.bar["ds_free", u].arrive()
            if put:
                self.bar["s_full"].arrive()

        return self.over_chunks(body, start, end)

    # ------------------------------------------------------------------ the hardware
    def step(self):
        """A load that lands, or the next step of a warp's products."""
        i = self.rnd.randrange(len(self.loads) + len(self.queues))
        if i < len(self.loads):
            buffer, n, name = self.loads.pop(i)
            self.holds[buffer] = n
            self.bar[name].landed(1)
            return
        queue = self.queues["QU"[i - len(self.loads)]]
        if not queue:
            return
        op = queue[0]
        if op[0] == "commit":
            self.bar[op[1]].arrive()
            queue.pop(0)
            return
        _, n, reads, writes, begun = op
        self.see(n, *reads)
        if not begun:
            for x in writes:
                self.holds[x] = None
            if "C" in writes:
                self.holds["P", 0] = self.holds["P", 1] = None
            op[4] = True
        else:
            for x in writes:
                self.holds[x] = n
            queue.pop(0)

    def run(self):
        roles = [self.plan(), self.tma(), self.mma_u()] + [f(h) for f in (self.tokens, self.state) for h in (0, 1)]
        if not self.local:
            roles += [self.mma_q(), self.rows(0), self.rows(1)]
        at = {r: None for r in roles}  # the barrier that each one waits at
        while at:
            if self.rnd.random() < 0.4:
                self.step()
                continue
            r = self.rnd.choice(list(at))
            try:
                at[r] = next(r)
            except StopIteration:
                del at[r]
                continue
            if at[r] is None or self.loads or any(self.queues.values()) or None in at.values():
                continue
            was = dict(at)  # all wait and nothing is under way: one more look of each
            for x in was:
                at[x] = next(x)
            if at == was:
                raise Stopped(str(sorted(map(str, was.values()))))
        while self.loads or any(self.queues.values()):
            self.step()
        assert self.ends == [len(self.units)] * 2


SHAPES = {
    "one": [1], "long": [7], "ones": [1] * 6, "mixed": [3, 1, 2, 5, 1],
    "empty": [0], "all_empty": [0] * 5, "empty_first": [0, 0, 0, 2], "empty_last": [2, 0, 0, 0],
    "empty_between": [1, 0, 0, 2, 0, 0, 0, 1], "alternating": [1, 0, 1, 0, 3, 0, 1],
}


@pytest.mark.parametrize("name", SHAPES)
def test_the_pipeline_ends_and_every_role_sees_its_chunk(name):
    for seed in range(60):
        Block(SHAPES[name], False, seed).run()


@pytest.mark.parametrize("name", ["one", "long", "ones", "mixed"])
def test_the_segments_own_states(name):
    for seed in range(60):
        Block(SHAPES[name], True, seed).run()


def test_random_units():
    rnd = random.Random(0)
    for seed in range(200):
        units = [rnd.choice([0, 0, 1, 1, 2, 3]) for _ in range(rnd.randint(1, 9))]
        Block(units, False, seed).run()


@pytest.mark.parametrize("name,stops", [("mixed", False), ("alternating", False), ("empty_first", False),
                                        ("empty_last", True), ("empty_between", True)])
def test_the_next_unit_before_the_last_q_stops_at_empty_units(name, stops):
    """The order that the kernel must not take: the ring has two places, and the units after an
    empty one appear only once every role has taken it, which they do only with that q."""
    for seed in range(20):
        if stops:
            with pytest.raises(Stopped):
                Block(SHAPES[name], False, seed, q_first=False).run()
        else:
            Block(SHAPES[name], False, seed, q_first=False).run()
