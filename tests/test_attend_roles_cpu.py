"""The barriers of the chunk attention's warps (csrc/paged_attn.cuh), as a model under
random schedules: every wait ends, none passes before its own phase or two phases late,
and the infinities and NaN of open rows that a part's rows read are that part's own.

The model has the kernel's rings, counts and parities, with three converting warps in
place of eight, one warp for each unit's softmax, and copies and products that complete
in order at random times."""
import random

import pytest

SLOTS, WARPS, NONE = 8, 3, (1 << 64) - 1


class Stuck(AssertionError):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.done = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending = self.count
            self.done += 1


def key(it, pos):
    return ((it ^ 0xffffffff) << 32) | pos


class Model:
    """parts: (tiles, whether units share them, position per converting warp of a value
    that is not finite or None). A plain flag, put back between parts, may take the place of
    the keys (`flag`), and a unit's rows may leave out that they have read them (`early`)."""

    def __init__(self, parts, stages, raws, seed, flag=False, early=False):
        self.parts, self.stages, self.raws, self.flag, self.early = parts, stages, raws, flag, early
        self.rng = random.Random(seed)
        self.bars, self.flight = {}, []
        for i in range(stages):
            self.bar("kv_full", i, WARPS), self.bar("kv_empty", i, 2)
        for i in range(raws):
            self.bar("raw_full", i, 1), self.bar("raw_empty", i, WARPS)
        for i in range(SLOTS):
            self.bar("info_full", i, 1), self.bar("info_empty", i, 2 + WARPS)
        for i in range(2):
            self.bar("s_full", i, 1), self.bar("p_full", i, 2), self.bar("o_done", i, 1)
            self.bar("fix_ready", i, WARPS), self.bar("fix_free", i, 2)
        self.bar("join_ready", 0, 2), self.bar("join_done", 0, 2), self.bar("conv", 0, WARPS)
        self.any, self.first = [0, 0], [NONE, NONE]

    def bar(self, name, i, count):
        self.bars[name, i] = Barrier(count)

    def arrive(self, name, i):
        self.bars[name, i].arrive()

    def later(self, name, i):
        self.flight.append((name, i))

    def wait(self, name, i, phase):
        """A wait for `phase`'s parity; -1 is the phase before the first."""
        b = self.bars[name, i]
        while (b.done & 1) == (phase & 1):
            yield
        assert phase < b.done <= phase + 1, "a wait for phase %d of %s passed after %d" % (phase, (name, i), b.done)

    @staticmethod
    def values(k, n, both):
        return k & 1 if both else int(k == 2 * n - 1 or (k > 0 and k % 2 == 0))

    @staticmethod
    def tile_of(k, n, both):
        return k >> 1 if both or k in (0, 2 * n - 1) else ((k + 1) >> 1 if k & 1 else (k >> 1) - 1)

    def tiles(self):
        i = x = 0

        def call():
            nonlocal x
            yield from self.wait("raw_empty", x % self.raws, x // self.raws - 1)
            self.later("raw_full", x % self.raws)
            x += 1
        for n, both, _ in self.parts:
            for j in range(n):
                yield from self.wait("info_empty", i % SLOTS, i // SLOTS - 1)
                self.arrive("info_full", i % SLOTS)
                yield
                yield from call()
                if both or j > 0:
                    yield from call()
                i += 1
            if not both:
                yield from call()

    def convert(self, w):
        before, conv = 0, 0
        for it, (n, both, bad) in enumerate(self.parts):
            par = it & 1
            yield from self.wait("fix_free", par, (it >> 1) - 1)
            if self.flag:
                yield
                if self.any[par]:
                    self.arrive("conv", 0)
                    yield from self.wait("conv", 0, conv)
                    self.any[par], self.first[par] = 0, NONE
                    self.arrive("conv", 0)
                    yield from self.wait("conv", 0, conv + 1)
                    conv += 2
            for k in range(2 * n):
                j, tile, i = self.tile_of(k, n, both), before + self.tile_of(k, n, both), 2 * before + k
                which = self.values(k, n, both)
                if not which:
                    yield from self.wait("info_full", tile % SLOTS, tile // SLOTS)
                yield from self.wait("raw_full", i % self.raws, i // self.raws)
                yield from self.wait("kv_empty", i % self.stages, i // self.stages - 1)
                for _ in range(self.rng.randrange(4)):
                    yield
                if which and j == n - 1 and bad[w] is not None:
                    self.first[par] = min(self.first[par], bad[w] if self.flag else key(it, bad[w]))
                    self.any[par] = it + 1
                self.arrive("kv_full", i % self.stages)
                self.arrive("raw_empty", i % self.raws)
                if which:
                    self.arrive("info_empty", tile % SLOTS)
                yield
            before += n
            self.arrive("fix_ready", par)

    def gate(self):
        x, opened = 0, [0, 0]

        def operand():
            nonlocal x
            yield from self.wait("kv_full", x % self.stages, x // self.stages)
            self.arrive("kv_empty", x % self.stages)
            x += 1
            yield

        def let(u):
            yield from self.wait("p_full", u, opened[u] - 1)
            opened[u] += 1
            self.arrive("p_full", u)
            yield
        for n, both, _ in self.parts:
            for _ in range(1 if both or n == 1 else 2):
                yield from operand()
            for j in range(n):
                yield from operand()
                if j + (1 if both else 2) < n:
                    yield from operand()
                for u in (0, 1) if both else (j & 1,):
                    yield from let(u)

    def products(self):
        x, phase = 0, [0, 0]

        def take():
            nonlocal x
            x += 1
            return x - 1

        def there(i):
            assert self.bars["kv_full", i % self.stages].done > i // self.stages, "products of an operand that is not there"

        def scores(u, i, last_use):
            there(i)
            self.later("s_full", u)
            if last_use:
                self.later("kv_empty", i % self.stages)
        for n, both, _ in self.parts:
            ahead = 1 if both else 2
            for u in range(2):
                if both and u:
                    scores(u, k, True)
                elif both or u < n:
                    yield from self.wait("kv_full", x % self.stages, x // self.stages)
                    k = take()
                    scores(u, k, not both)
                yield
            for j in range(n):
                more, v = j + ahead < n, take()
                k = take() if more else None
                units = (0, 1) if both else (j & 1,)
                for u in units:
                    yield from self.wait("p_full", u, phase[u])
                    phase[u] += 1
                    there(v)
                    if u == units[-1]:
                        self.later("kv_empty", v % self.stages)
                    if more:
                        scores(u, k, u == units[-1])
                    else:
                        self.later("o_done", u)
                    yield

    def softmax(self, u):
        t, scores, outs, joins = 0, 0, [0, 0], 0
        for it, (n, both, bad) in enumerate(self.parts):
            par = it & 1
            for j in range(n):
                yield from self.wait("info_full", t % SLOTS, t // SLOTS)
                if both or (j & 1) == u:
                    yield from self.wait("s_full", u, scores)
                    scores += 1
                    for _ in range(self.rng.randrange(4)):
                        yield
                    self.arrive("p_full", u)
                self.arrive("info_empty", t % SLOTS)
                t += 1
                yield
            if self.early:
                self.arrive("fix_free", par)
            yield from self.wait("fix_ready", par, it >> 1)
            has = (True, both or n > 1)
            for v in (u,) if both else (0, 1):
                if has[v]:
                    yield from self.wait("o_done", v, outs[v])
            if not both:
                self.arrive("join_ready", 0)
                yield from self.wait("join_ready", 0, joins)
            yield
            want = min([p for p in bad if p is not None], default=None)
            got = self.any[par] != 0 if self.flag else self.any[par] == it + 1
            assert got == (want is not None), "part %d takes the marks of another" % it
            if got:
                assert self.first[par] == (want if self.flag else key(it, want)), "part %d takes a position of another" % it
            if not both:
                self.arrive("join_done", 0)
                yield from self.wait("join_done", 0, joins)
                joins += 1
            outs = [o + h for o, h in zip(outs, has)]
            if not self.early:
                self.arrive("fix_free", par)
            yield

    def run(self):
        live = [self.tiles(), self.gate(), self.products(), self.softmax(0), self.softmax(1)]
        live += [self.convert(w) for w in range(WARPS)]
        rng, idle = self.rng, 0
        while live:
            if self.flight and rng.random() < 0.4:  # copies complete in order, and so do products
                copy = rng.random() < 0.5
                i = next((i for i, f in enumerate(self.flight) if (f[0] == "raw_full") == copy), None)
                if i is not None:
                    self.arrive(*self.flight.pop(i))
            role = rng.choice(live)
            state = [(b.done, b.pending) for b in self.bars.values()]
            for _ in range(rng.choice([1, 1, 5, 40])):
                try:
                    next(role)
                except StopIteration:
                    live.remove(role)
                    break
            moved = state != [(b.done, b.pending) for b in self.bars.values()]
            idle = 0 if moved or self.flight else idle + 1
            if idle > 2000:
                raise Stuck("no role goes on")


def some_parts(rng, bad):
    def mark():
        return rng.randrange(100) if rng.random() < 0.6 else None
    return [(rng.choice([1, 1, 1, 2, 3, 4, 5, 9]), rng.random() < 0.5,
             [mark() for _ in range(WARPS)] if rng.random() < bad else [None] * WARPS) for _ in range(rng.randrange(1, 10))]


@pytest.mark.parametrize("stages,raws", [(3, 3), (6, 6)])  # 128 and 64 channels
@pytest.mark.parametrize("bad", [0.0, 0.4, 1.0])
def test_every_wait_ends_and_is_for_its_own_phase(stages, raws, bad):
    for seed in range(40):
        Model(some_parts(random.Random(seed), bad), stages, raws, seed).run()


def test_the_model_finds_a_barrier_behind_a_flag_that_its_own_part_may_set():
    """A warp that comes to the part's start late would take the others' mark of this part
    for one of the part before, and wait for them at a barrier to which none of them comes."""
    found = 0
    for seed in range(40):
        try:
            Model(some_parts(random.Random(seed), 1.0), 3, 3, seed, flag=True).run()
        except AssertionError:
            found += 1
    assert found > 0


def test_the_model_finds_marks_that_are_overwritten_before_they_are_read():
    found = 0
    for seed in range(40):
        try:
            Model(some_parts(random.Random(seed), 0.5), 6, 6, seed, early=True).run()
        except AssertionError:
            found += 1
    assert found > 0
