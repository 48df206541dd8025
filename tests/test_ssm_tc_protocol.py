"""CPU model of the tcgen05 scan's hand-over protocol (no GPU).

A block of ssm_tc_kernel (ssm_tc.cu) has warps that load tiles, form decays,
decay scores into P, advance the state, form addends and issue the matrix
products, synchronised by mbarriers whose waits name a phase by its parity.
Products run behind their issue. A commit's barrier is signalled once every
product issued before it has completed; products with the same accumulator
complete in the order of their issue, others in any order. Nothing else orders a
product with respect to another one or to a warp that writes what it reads. And a
commit speaks for products only: copies, and what a warp wrote or has read itself,
are known to those who wait for a barrier on which the copy or the warp arrived, or
another warp that knew of it.

The order in which the product warp waits, issues, commits and arrives is read from
the kernel's source; the other roles are written out with its index and parity
formulas. All are interleaved at random, with some of the warps held back and with products
and copies that complete late. Whatever is read must hold the chunk it is meant to and
be known to the reader, nothing may be written while a product or a copy in flight reads or writes it, every wait
that passes must be for the phase it meant, and every warp must finish.
"""
import functools
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_104_b200", "csrc", "ssm_tc.cu")
W_PLACES = 5
LATE = (0.004, 0.05, 0.5)  # how often a product or copy completes rather than a warp moves on


def product_steps():
    """What the product warp does in a chunk, in the order of the source: ("wait", barrier, phase, not in the first
    chunk), ("issue", product), ("update", first, last), ("commit", barrier), ("arrive", barrier)."""
    with open(SOURCE, encoding="utf-8") as f:
        text = f.read()
    kernel = text[text.index("ssm_tc_kernel("):text.index("ssm_tc_ends_kernel(")]
    part = kernel[kernel.index("for (int c = 0; c < n_chunks; ++c)"):]
    part = re.sub(r"//[^\n]*", "", part[:part.index("if (!ok)")])
    a, z = part.index("auto update ="), part.index("return true;")
    update = part[a:z]  # of 16 tokens: wait for their addends, the products, the place handed back
    order = [update.index(s) for s in ("wait_warp(&bars[W_FULL + place]", "mma_ts_f16_by(lead, tb + T_S", "mma_commit_by(lead, &bars[W_FREE + place]")]
    assert order == sorted(order)
    part = part[z + len("return true;"):]
    pattern = (r"(?P<first>c == 0 \|\| )?wait_warp\(&bars\[(?P<wait>\w+)(?: \+ par)?\], (?P<phase>par2|par|\(c - 1\) & 1), abort\)"
               r"|over_columns\(tb \+ (?P<over>T_G|T_Y)|update\((?P<lo>\w+), (?P<hi>\w+)\)|mma_ts_f16_by\(lead, tb \+ (?P<px>T_Y)"
               r"|mma_commit_by\(lead, &bars\[(?P<commit>\w+)(?: \+ par)?\]\)|mbar_arrive_by\(lead, &bars\[(?P<arrive>\w+)\]\)")
    number = {"W_PLACES": W_PLACES, "0": 0, "8": 8}
    steps = []
    for m in re.finditer(pattern, part):
        if m["wait"]:
            steps.append(("wait", m["wait"], m["phase"], bool(m["first"])))
        elif m["over"]:
            steps.append(("issue", "G" if m["over"] == "T_G" else "CS"))
        elif m["lo"]:
            steps.append(("update", number[m["lo"]], number[m["hi"]]))
        elif m["px"]:
            steps.append(("issue", "PX"))
        elif m["commit"]:
            steps.append(("commit", m["commit"]))
        else:
            steps.append(("arrive", m["arrive"]))
    assert [s[1] for s in steps if s[0] == "issue"] == ["G", "CS", "PX"]
    assert [s[1:] for s in steps if s[0] == "update"] == [(0, W_PLACES), (W_PLACES, 8)]
    assert len(re.findall(r"wait_warp\(", part)) == sum(s[0] == "wait" for s in steps)
    assert len(re.findall(r"mma_commit_by\(", part)) == sum(s[0] == "commit" for s in steps)
    return steps


@functools.cache
def zeroing_waits():
    """What a warp of the addends waits for before it zeroes b behind the segment, in the last chunk."""
    with open(SOURCE, encoding="utf-8") as f:
        text = f.read()
    text = text[text.index("ssm_tc_kernel("):]
    return re.findall(r"wait_warp\(&bars\[(\w+)", re.search(r"if \(m < Q && ([^\n]*)", text)[1])


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0
        self.known = set()  # what who waits for it learns

    def arrive(self, known=()):
        self.pending -= 1
        self.known |= set(known)
        assert self.pending >= 0
        if self.pending == 0:
            self.done += 1
            self.pending = self.count

    def passes(self, parity):
        return (self.done & 1) != parity


class Block:
    def __init__(self, steps, chunks, nh, nxq, seed):
        self.steps, self.chunks, self.nh, self.nxq = steps, chunks, nh, nxq
        self.rng = random.Random(seed)
        one = ["C_FULL", "C_FREE", "G_DONE", "Y2_DONE", "Y_DONE", "ST_DONE"]
        self.bars = {k: Barrier(1 + steps.count(("arrive", k))) for k in one}
        self.bars |= {k: Barrier(4) for k in ("S_READY", "YS_READY")} | {k: Barrier(8) for k in ("P_READY", "Y_FREE")}
        for k in range(2):
            self.bars |= {("B_FULL", k): Barrier(1), ("B_FREE", k): Barrier(1), ("SC_FULL", k): Barrier(nh), ("SC_FREE", k): Barrier(20)}
        self.bars |= {("W_FULL", k): Barrier(4) for k in range(W_PLACES)} | {("W_FREE", k): Barrier(1) for k in range(W_PLACES)}
        self.bars |= {("X_FULL", k): Barrier(1) for k in range(nxq)} | {("X_FREE", k): Barrier(2) for k in range(nxq)}
        self.holds = {}      # place -> what lies there
        self.flying = []     # products in flight: dict(acc, reads, writes, finish)
        self.copies = []     # (place, content, barrier) on the way to shared memory, (place, None, None) on the way out
        self.commits = []    # (products that it waits for, barrier)

    # ---- memory

    def read(self, place, want):
        assert not any(place in p["writes"] for p in self.flying), ("read while a product writes", place)
        assert not any(c[0] == place and c[1] for c in self.copies), ("read while a copy writes", place)
        assert self.holds.get(place) == want, (place, self.holds.get(place), want)

    def write(self, place, what):
        assert not any(place in p["writes"] or place in p["reads"] for p in self.flying), ("written under a product", place)
        assert not any(c[0] == place for c in self.copies), ("written under a copy", place)
        self.holds[place] = what

    def issue(self, acc, reads, results):
        """A product: `reads` place -> content it needs, `results` place -> content it leaves."""
        for place, want in reads.items():
            assert self.holds.get(place) == want, (acc, place, self.holds.get(place), want)
        for p in self.flying:
            if p["acc"] == acc:
                continue
            clash = p["writes"] & (reads.keys() | results.keys()) | p["reads"] & results.keys()
            assert not clash, (acc, "issued over", p["acc"], sorted(clash, key=str)[0])
        self.flying.append(dict(acc=acc, reads=set(reads), writes=set(results)))
        self.holds.update(results)

    def commit(self, bar):
        self.commits.append(([id(p) for p in self.flying], bar))
        self.settle()

    def settle(self):
        live = {id(p) for p in self.flying}
        rest = []
        for ids, bar in self.commits:
            ids = [i for i in ids if i in live]
            if ids:
                rest.append((ids, bar))
            else:
                self.bars[bar].arrive()
        self.commits = rest

    def background(self):
        """One product or copy completes."""
        ready = [p for k, p in enumerate(self.flying) if not any(q["acc"] == p["acc"] for q in self.flying[:k])]
        k = self.rng.randrange(len(ready) + len(self.copies))
        if k < len(ready):
            self.flying.remove(ready[k])
            self.settle()
        else:
            place, what, bar = self.copies.pop(k - len(ready))[:3]
            if bar is not None:
                self.holds[place] = what
                self.bars[bar].arrive([(place[0], what)])

    def wait(self, bar, parity, phase, known=None):
        while not self.bars[bar].passes(parity):
            yield
        assert self.bars[bar].done == phase, (bar, self.bars[bar].done, phase)
        if known is not None:
            known |= self.bars[bar].known

    def load(self, place, what, bar):
        assert not any(place in p["reads"] for p in self.flying) and not any(c[0] == place for c in self.copies), place
        self.copies.append((place, what, bar))

    # ---- roles

    def loader(self):
        nb = nx = nc = 0
        while nb < self.chunks or nc < self.chunks or nx < 4 * self.chunks:
            if nb < self.chunks and (nb < 2 or self.bars["B_FREE", nb & 1].passes((nb // 2 - 1) & 1)):
                self.load(("b", nb & 1), nb, ("B_FULL", nb & 1))
                nb += 1
            if nc < self.chunks and (nc < 1 or self.bars["C_FREE"].passes((nc - 1) & 1)):
                self.load("c", nc, "C_FULL")
                nc += 1
            xp = nx % self.nxq
            if nx < 4 * self.chunks and (nx < self.nxq or self.bars["X_FREE", xp].passes((nx // self.nxq - 1) & 1)):
                if nx >= self.nxq:
                    known = self.bars["X_FREE", xp].known
                    assert all(("taken", nx - self.nxq, q, h) in known for q in range(4) for h in (0, 1)), "x loaded over its readers"
                self.load(("x", xp), nx, ("X_FULL", xp))
                nx += 1
            yield

    def step_sizes(self, h):
        for c in range(self.chunks):
            if c >= 2:
                yield from self.wait(("SC_FREE", c & 1), (c // 2 - 1) & 1, c // 2)
            self.holds["scalars", c & 1, h] = c
            self.bars["SC_FULL", c & 1].arrive()
            yield

    def scalars(self, c, heads):
        for h in heads:
            assert self.holds["scalars", c & 1, h] == c

    def scores(self, quad, half):
        stored, known = [], set()
        for c in range(self.chunks):
            yield from self.wait(("SC_FULL", c & 1), (c // 2) & 1, c // 2 + 1)
            yield from self.wait("G_DONE", c & 1, c + 1)
            self.scalars(c, range(self.nh))
            self.read(("g", quad, half), ("scores", c))
            yield
            self.write(("g", quad, half), ("decayed", c))
            self.bars["P_READY"].arrive()
            if c > 0:
                while any(s in self.copies for s in stored):  # its stores have read x's place
                    yield
                stored = []
                self.bars["X_FREE", (4 * (c - 1) + quad) % self.nxq].arrive(known)
            yield from self.wait("Y_DONE", c & 1, c + 1, known)
            self.read("y", ("whole", c))
            place = ("x", (4 * c + quad) % self.nxq)
            assert self.holds[place] == 4 * c + quad and ("x", 4 * c + quad) in known, "x read without a word of its copy"
            for q in range(4):
                for h in (0, 1):
                    assert self.holds["flags", c % 3, q, h] == c and ("flags", c, q, h) in known, "flags read without a word of them"
            assert not any(place in p["reads"] for p in self.flying), "x overwritten under a product"
            yield
            self.bars["Y_FREE"].arrive()
            stored.append((place, None, None, quad, half, c))
            self.copies.append(stored[-1])
            self.bars["SC_FREE", c & 1].arrive()
            yield

    def state(self, quad):
        for c in range(self.chunks):
            yield from self.wait(("SC_FULL", c & 1), (c // 2) & 1, c // 2 + 1)
            self.scalars(c, range(self.nh))
            if c > 0:
                yield from self.wait("ST_DONE", (c - 1) & 1, c)
                self.read("s", ("updated", c - 1))
            self.write(("rounded", quad), c)
            yield
            self.write(("s", quad), ("decayed", c))
            self.bars["S_READY"].arrive()
            self.bars["SC_FREE", c & 1].arrive()
            yield from self.wait("Y2_DONE", c & 1, c + 1)
            self.read("y", ("read", c))
            self.write(("y", quad), ("scaled", c))
            self.bars["YS_READY"].arrive()
            yield

    def addends(self, quad, half):
        known = set()
        for c in range(self.chunks):
            yield from self.wait(("SC_FULL", c & 1), (c // 2) & 1, c // 2 + 1)
            self.scalars(c, range(self.nh))
            if c == self.chunks - 1:
                assert set(zeroing_waits()) <= {"B_FULL", "G_DONE"}
                if "B_FULL" in zeroing_waits():
                    yield from self.wait(("B_FULL", c & 1), (c // 2) & 1, c // 2 + 1, known)
                if "G_DONE" in zeroing_waits():
                    yield from self.wait("G_DONE", c & 1, c + 1)
                assert ("b", c) in known, "b zeroed before it came"
            for q in range(4):
                nx = 4 * c + q
                nw = 2 * nx + half
                place = nw % W_PLACES
                yield from self.wait(("X_FULL", nx % self.nxq), (nx // self.nxq) & 1, nx // self.nxq + 1, known)
                assert ("x", nx) in known
                self.read(("x", nx % self.nxq), nx)
                known.add(("taken", nx, quad, half))
                if c == self.chunks - 1:
                    assert self.bars["G_DONE"].done == c + 1, "b zeroed while the scores may read it"
                if nw >= W_PLACES:
                    yield from self.wait(("W_FREE", place), (nw // W_PLACES - 1) & 1, nw // W_PLACES)
                self.write(("w", place, quad), nw)
                self.holds["flags", c % 3, quad, half] = c
                known.add(("flags", c, quad, half))
                if q == 3:
                    self.bars["SC_FREE", c & 1].arrive()
                self.bars["W_FULL", place].arrive(known)
                yield

    def products(self):
        quads, known = range(4), set()
        for c in range(self.chunks):
            for step in self.steps:
                if step[0] == "wait":
                    _, name, phase, not_first = step
                    if not_first and c == 0:
                        continue
                    bar = (name, c & 1) if name == "B_FULL" else name
                    yield from self.wait(bar, {"par": c & 1, "par2": (c // 2) & 1}.get(phase, (c - 1) & 1),
                                         {"par": c + 1, "par2": c // 2 + 1}.get(phase, c))
                elif step == ("issue", "G"):
                    self.issue("g", {"c": c, ("b", c & 1): c}, {("g", q, h): ("scores", c) for q in quads for h in (0, 1)})
                elif step == ("issue", "CS"):
                    self.issue("y", {"c": c} | {("rounded", q): c for q in quads}, {"y": ("read", c)})
                elif step == ("issue", "PX"):
                    self.issue("y", {("g", q, h): ("decayed", c) for q in quads for h in (0, 1)} |
                               {("y", q): ("scaled", c) for q in quads} | {("x", (4 * c + q) % self.nxq): 4 * c + q for q in quads},
                               {"y": ("whole", c)})
                elif step[0] == "update":
                    for g in range(step[1], step[2]):
                        nw = 8 * c + g
                        place = nw % W_PLACES
                        yield from self.wait(("W_FULL", place), (nw // W_PLACES) & 1, nw // W_PLACES + 1, known)
                        self.issue("s", {("w", place, q): nw for q in quads} | {("b", c & 1): c} | {("s", q): ("decayed", c) for q in quads},
                                   {"s": ("updated", c)})
                        yield
                        self.commit(("W_FREE", place))
                elif step[0] == "arrive":
                    self.bars[step[1]].arrive(known)
                else:
                    self.commit((step[1], c & 1) if step[1] == "B_FREE" else step[1])
                yield

    def run(self, late):
        live = [self.loader(), self.products()] + [self.step_sizes(h) for h in range(self.nh)]
        live += [self.scores(q, h) for q in range(4) for h in (0, 1)] + [self.state(q) for q in range(4)]
        live += [self.addends(q, h) for q in range(4) for h in (0, 1)]
        slow = set(map(id, self.rng.sample(live, 6)))  # (these seldom get a turn)
        for _ in range(2_000_000):
            if (self.flying or self.copies) and (not live or self.rng.random() < late):
                self.background()
            elif live:
                w = self.rng.choice(live)
                if id(w) in slow and self.rng.random() < 0.99:
                    continue
                try:
                    next(w)
                except StopIteration:
                    live.remove(w)
            else:
                return
        raise AssertionError("no progress")


@pytest.mark.parametrize("nh,nxq", [(1, 11), (2, 11), (1, 8), (2, 8)])
def test_every_tile_is_handed_over_whole_in_any_order(nh, nxq):
    steps = product_steps()
    for seed in range(12):
        Block(steps, 1 + 3 * (seed % 3), nh, nxq, seed).run(late=LATE[seed // 4])


@pytest.mark.parametrize("barrier", ["C_FULL", "B_FULL", "Y_DONE", "S_READY", "Y_FREE", "P_READY", "YS_READY"])
def test_the_model_notices_each_wait_that_is_left_out(barrier):
    """Each of the product warp's waits taken out (of the model) is found."""
    steps = [s for s in product_steps() if s[:2] != ("wait", barrier)]
    with pytest.raises(AssertionError):
        for seed in range(24):
            Block(steps, 7, 1, 11, seed).run(late=LATE[seed % 3])


def test_the_model_notices_an_arrival_that_is_left_out():
    """What the product warp passes on beside its commits."""
    steps = [s for s in product_steps() if s[0] != "arrive"]
    with pytest.raises(AssertionError, match="without a word"):
        Block(steps, 2, 1, 11, 0).run(late=0.5)


@pytest.mark.parametrize("kernel", ["ssm_tc_kernel(", "ssm_tc_ends_kernel("])
def test_every_barrier_is_set_up_once(kernel):
    """One mbarrier.init each: on a barrier that has been set up, a second one is undefined."""
    with open(SOURCE, encoding="utf-8") as f:
        text = f.read()
    text = text[text.index(kernel):]
    setup = text[:text.index("tc::mbar_init_fence()")]
    setup = setup[setup.rindex("    if (tid "):]
    assert len(re.findall(r"\binit\(|mbar_init\(", setup)) == 1 and "for (" not in setup
    assert setup.lstrip().startswith("if (tid < BARS) {") and "const int b = tid;" in setup and "mbar_init(&bars[b]," in setup
