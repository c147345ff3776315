"""The rings of the 16-bit cache's attention kernels, walked through by random interleavings of their roles (no GPU needed).

A model of cp_kv16_prompt.cu (copies, two MMA warps, the look over the values, two warpgroups of rows; copies and MMAs finish
later, in any order that the hardware allows) and of cp_kv16_attention.cu (copies, four warps).  Checked on every
step: a wait by parity passes in the phase it means and in no other, no barrier counts past its end, a stage is read
only while the tile it should hold lies in it and written only once it is free, and all roles end.  With a copy
that is never made, or a wait that gives up at a random moment, all roles end too, and no copy or MMA is in flight then."""
import random

import pytest

LIMIT = 3000  # clocks that a wait lasts


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than a phase has"
        self.pending -= 1
        self.tx += tx
        self.check()

    def land(self, n):
        self.tx -= n
        self.check()

    def check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count


class GaveUp(Exception):
    pass


class Walk:
    """Clock, barriers, copies in flight and the roles of one CTA."""

    def __init__(self, seed, quit_at=None):
        self.R, self.clock, self.later, self.abort = random.Random(seed), 0, [], False
        self.bars, self.stage, self.roles, self.quit_at = {}, {}, {}, quit_at

    def bar(self, name, count):
        self.bars[name] = Bar(count)

    def wait(self, role, name, phase):
        """kv16_wait: passes when the parity says so, gives up with the others or at its limit."""
        b, since = self.bars[name], self.clock
        while (b.phase & 1) == (phase & 1):
            if self.abort or self.clock - since > LIMIT or (self.quit_at is not None and self.quit_at[0] == role and self.clock > self.quit_at[1]):
                self.abort = True
                raise GaveUp
            yield
        assert b.phase == phase + 1, ("a wait passed in another phase", name, phase, b.phase)

    def copy(self, ring, st, k, full):
        old = self.stage.get((ring, st))
        assert old is None or old[1] == "free", ("a stage is written before it is free", ring, k, old)
        self.stage[ring, st] = [k, "loading"]
        self.bars[full].arrive(1)

        def land():
            self.stage[ring, st][1] = "there"
            self.bars[full].land(1)

        self.later.append((self.clock + self.R.choice([1, 3, 10, 60, 200]), land))

    def tick(self):
        self.clock += 1
        for x in [x for x in self.later if x[0] <= self.clock]:
            self.later.remove(x)
            x[1]()

    def run(self, roles, always=()):
        """All roles to their end, at random speeds; `always` runs beside them."""
        names = list(roles) + [r for r, _ in always]
        both = {**roles, **dict(always)}
        speed = {r: self.R.choice([1, 1, 3, 10]) for r in names}
        live = set(roles)
        while live:
            self.tick()
            self.R.shuffle(names)
            for r in names:
                if (r in live or r not in roles) and not self.R.randrange(speed[r]):
                    try:
                        next(both[r])
                    except (StopIteration, GaveUp):
                        live.discard(r)
            assert self.clock < 50 * LIMIT, ("roles that do not end", live)

    def drain(self, rings, copied):
        """After the last barrier of the CTA, where something gave up: the newest copy of each stage is waited for."""
        for ring, stages, full in rings:
            for k in range(max(0, copied[ring] - stages), copied[ring]):
                while (self.bars[full, k % stages].phase & 1) == (k // stages & 1):
                    self.tick()
                    assert self.clock < 100 * LIMIT


def item(pair, it, n):
    """prompt_item: (values?, tile) at place `it` of 2 n."""
    if pair:
        return bool(it & 1), it >> 1
    if it == 2 * n - 1:
        return True, n - 1
    if it == 0 or it & 1:
        return False, (it + 1) >> 1
    return True, (it >> 1) - 1


def prompt(pair, ST, n, seed, items=None, quit_at=None, late_drain=True):
    W = Walk(seed, quit_at)
    R = W.R
    for i in range(ST):
        for x in "kv":
            W.bar((x + "full", i), 1)
            W.bar((x + "empty", i), 2 if pair else 1)
        W.bar(("clean", i), 1)
    for w in range(2):
        for x in ("sfull", "ohalf", "oend"):
            W.bar((x, w), 1)
        for half in range(2):
            W.bar(("pready", w, half), 1)
    held, queue, frees, copied = {}, {0: [], 1: []}, {}, {"k": 0, "v": 0}

    def copies():
        gave_up = False
        for it in range(2 * n if items is None else items):
            v, k = item(pair, it, n)
            x = "kv"[v]
            if it >= 3 and k >= ST:
                try:
                    yield from W.wait("copies", (x + "empty", k % ST), k // ST - 1)
                except GaveUp:
                    gave_up = True
                    break
            if x == "k":
                held[k % 8] = k
            W.copy(x, k % ST, k, (x + "full", k % ST))
            copied[x] += 1
            yield
        if gave_up and not late_drain:
            for x in "kv":
                for k in range(max(0, copied[x] - ST), copied[x]):
                    while (W.bars[x + "full", k % ST].phase & 1) == (k // ST & 1):
                        yield

    def mma(w):
        q = queue[w]

        def scores(k):
            q.extend([("mma", "k", k), ("commit", ("sfull", w)), ("commit", ("kempty", k % ST))])

        def issue():
            first = 0 if pair else w
            if first < n:
                yield from W.wait(f"mma{w}", ("kfull", first % ST), first // ST)
                scores(first)
            t = 0
            while True:
                k, following = (t, t + 1) if pair else (2 * t + w, 2 * t + w + 2)
                if k >= n:
                    return
                yield from W.wait(f"mma{w}", ("clean", k % ST), k // ST)
                for half in range(2):
                    yield from W.wait(f"mma{w}", ("pready", w, half), t)
                    q.append(("mma", "v", k))
                    if half == 0:
                        q.append(("commit", ("ohalf", w)))
                        if following < n:
                            yield from W.wait(f"mma{w}", ("kfull", following % ST), following // ST)
                    yield
                q.append(("commit", ("vempty", k % ST)))
                if following < n:
                    scores(following)
                else:
                    q.append(("commit", ("oend", w)))
                t += 1

        try:
            yield from issue()
        except GaveUp:
            pass
        while q:  # every MMA issued completes before the CTA ends
            yield

    def tensor_cores():
        while True:
            ready = [w for w in range(2) if queue[w]]
            if not ready:
                yield
                continue
            w = R.choice(ready)
            op = queue[w][0]
            if op[0] == "mma":
                _, x, k = op
                for _ in range(R.choice([1, 2, 5])):
                    assert W.stage[x, k % ST] == [k, "there"], ("an MMA reads what is not there", x, k, W.stage[x, k % ST])
                    yield
            else:
                name = op[1]
                if name[0] in ("kempty", "vempty"):
                    key = (name[0][0], name[1])
                    frees[key] = frees.get(key, 0) + 1
                    if frees[key] == (2 if pair else 1):
                        frees[key] = 0
                        W.stage[key][1] = "free"
                W.bars[name].arrive()
                yield
            queue[w].pop(0)

    def look():
        for k in range(n):
            yield from W.wait("look", ("vfull", k % ST), k // ST)
            assert held[k % 8] == k
            for _ in range(R.choice([0, 0, 5, 100])):
                yield
            W.bars["clean", k % ST].arrive()
            yield

    def rows(w):
        t = 0
        while (t if pair else 2 * t + w) < n:
            k = t if pair else 2 * t + w
            yield from W.wait(f"rows{w}", ("sfull", w), t)
            assert held[k % 8] == k
            for half in range(2):
                for _ in range(R.choice([1, 5, 40])):
                    yield
                if half == 1 and R.random() < 0.3:
                    yield from W.wait(f"rows{w}", ("ohalf", w), t)
                W.bars["pready", w, half].arrive()
                yield
            t += 1
        if t:
            yield from W.wait(f"rows{w}", ("oend", w), 0)

    W.run({"copies": copies(), "mma0": mma(0), "mma1": mma(1), "look": look(), "rows0": rows(0), "rows1": rows(1)},
          [("tensor cores", tensor_cores())])
    if W.abort and late_drain:
        W.drain([("k", ST, "kfull"), ("v", ST, "vfull")], copied)
    assert not any(s[1] == "loading" for s in W.stage.values()), "a copy in flight at the end"
    assert not queue[0] and not queue[1]
    return W.abort


def few(ST, n, seed, items=None, quit_at=None, late_drain=True):
    W = Walk(seed, quit_at)
    for i in range(ST):
        W.bar(("full", i), 1)
        W.bar(("empty", i), 4)
    copied, readers = {"kv": 0}, {}

    def copies():
        for k in range(n if items is None else items):
            if k >= ST:
                yield from W.wait("copies", ("empty", k % ST), k // ST - 1)
            W.copy("kv", k % ST, k, ("full", k % ST))
            copied["kv"] += 1
            yield

    def rows(w):
        for k in range(n):
            yield from W.wait(f"rows{w}", ("full", k % ST), k // ST)
            for _ in range(W.R.choice([1, 3, 30])):
                assert W.stage["kv", k % ST] == [k, "there"], "rows read what is not there"
                yield
            readers[k] = readers.get(k, 0) + 1
            if readers[k] == 4:
                W.stage["kv", k % ST][1] = "free"
            W.bars["empty", k % ST].arrive()
            yield

    W.run({"copies": copies(), **{f"rows{w}": rows(w) for w in range(4)}})
    if W.abort and late_drain:
        W.drain([("kv", ST, "full")], copied)
    assert not any(s[1] == "loading" for s in W.stage.values()), "a copy in flight at the end"
    return W.abort


SIZES = list(range(1, 12)) + [25]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("stages", [2, 4])
def test_prompt_rings(pair, stages):
    for n in SIZES:
        for seed in range(12):
            assert not prompt(pair, stages, n, 7919 * seed + n)


@pytest.mark.parametrize("stages", [3, 6])
def test_few_row_ring(stages):
    for n in SIZES:
        for seed in range(12):
            assert not few(stages, n, 7919 * seed + n)


@pytest.mark.parametrize("missing", ["last", "all"])
def test_roles_end_without_a_copy(missing):
    for n in (1, 2, 3, 6):
        for seed in range(3):
            for pair in (False, True):
                for stages in (2, 4):
                    assert prompt(pair, stages, n, seed, items=2 * n - 1 if missing == "last" else 0)
            for stages in (3, 6):
                assert few(stages, n, seed, items=n - 1 if missing == "last" else 0)


ROLES = ["copies", "mma0", "mma1", "look", "rows0", "rows1"]


def _quits(late_drain):
    """Walks in which one role's wait gives up at a random moment: how many did, how many left a copy in flight."""
    gave, left = 0, 0
    for seed in range(240):
        r = random.Random(seed)
        n, at = r.choice([2, 5, 9, 14]), r.randrange(0, 400)
        try:
            if seed % 4:
                gave += prompt(bool(seed & 1), r.choice([2, 4]), n, seed, quit_at=(r.choice(ROLES), at), late_drain=late_drain)
            else:
                gave += few(r.choice([3, 6]), n, seed, quit_at=(r.choice(["copies", "rows0", "rows2"]), at), late_drain=late_drain)
        except AssertionError as e:
            assert str(e).startswith("a copy in flight at the end"), e
            left += 1
    return gave, left


def test_nothing_is_in_flight_after_a_wait_that_gave_up():
    gave, left = _quits(True)
    assert left == 0 and gave > 60


def test_the_copying_warp_alone_does_not_know():
    """Copies waited for only where the copying warp's own wait gave up: others may give up after it is through."""
    assert _quits(False)[1] > 0
