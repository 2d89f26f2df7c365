"""The prompt attention's barriers as a model on the CPU: copies and products that finish in any order.  Every wait by parity
must pass only when its own phase is complete, and a product may read a tile only while it holds what the product takes.
Waits may also give up, as the kernel's do after their time limit: every role ends all the same, and not before its copies
and products have.

The places of the ring come from the kernel's own header; the roles (copies, S, P V, the check of V, the rows of two tiles)
go through the waits and arrivals of the kernel in their order."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PART = 3    # tiles of keys that a pair's rows may see only in part
SLOTS = 2
LANDS = "a wait of a role that gave up, for what it started: it has to come"
LONG = "a wait for what no role is needed for: it gives up only when nothing goes on"


class Stale(AssertionError):
    """A wait passed, or a product began, before its time."""


class Barrier:
    """An mbarrier: `count` arrivals and the bytes expected (copies, here) complete a phase."""

    def __init__(self, count=1):
        self.count, self.phase, self.pending, self.tx = count, 0, count, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        self._turn()

    def expect(self, n):
        self.tx += n
        self.arrive()

    def landed(self):
        self.tx -= 1
        assert self.tx >= 0
        self._turn()

    def passes(self, phase):
        """try_wait.parity for that phase; it must be complete, not one that lies ahead of the present one."""
        if self.phase & 1 == phase & 1:
            return False
        if self.phase <= phase:
            raise Stale(f"a wait for phase {phase} passed in phase {self.phase}")
        return True


class Tile:
    def __init__(self):
        self.holds, self.readers = None, 0


class Model:
    """items: (tiles of A, tiles of B, first tile seen in part).  ring: stage, full, parity by use.  gives_up: how likely a
    wait is to end without its phase."""

    def __init__(self, items, stages, ring, rng, gives_up=0.0):
        self.items, self.stages, self.ring, self.rng, self.gives_up = items, stages, ring, rng, gives_up
        two = lambda n=1: [Barrier(n) for _ in range(SLOTS)]  # noqa: E731
        self.item_full, self.item_empty = two(), two(11)
        self.next, self.q_full, self.q_empty = Barrier(), Barrier(), Barrier()
        self.full, self.empty = [Barrier() for _ in range(2 * stages)], [Barrier() for _ in range(stages)]
        self.s_full, self.s_taken, self.p_full, self.pv_done = two(), Barrier(4), two(4), two()
        self.rows_done, self.drained = two(4), {"S": Barrier(), "PV": Barrier()}
        self.go, self.checked = [[Barrier() for _ in range(PART)] for _ in range(SLOTS)], [[Barrier() for _ in range(PART)] for _ in range(SLOTS)]
        self.tiles, self.q = [Tile() for _ in range(stages)], Tile()
        self.slot = [None] * SLOTS
        self.copies = []                      # in flight: (kind, action)
        self.queue = {"S": [], "PV": []}      # products of a warp, in order
        self.outputs = []

    # ---- what is asynchronous
    def copy(self, kind, tile, what, bar):
        if tile.readers:
            raise Stale("a copy into a tile that is being read")
        tile.holds = None

        def land():
            tile.holds = what
            bar.landed()
        self.copies.append((kind, land))

    def product(self, warp, reads):
        for tile, what in reads:
            if tile.holds != what:
                raise Stale(f"{warp} of {what} from a tile that holds {tile.holds}")
            tile.readers += 1

        def done():
            for tile, what in reads:
                if tile.holds != what:
                    raise Stale("a tile was overwritten under a product")
                tile.readers -= 1
        self.queue[warp].append(done)

    def commit(self, warp, bar):
        self.queue[warp].append(bar.arrive)

    # ---- the roles; each yields (barrier, phase) that it waits for, and is told whether it gave up
    def take(self, t):
        return (yield self.item_full[t % 2], t // 2)

    def load(self):
        use = n_q = t = 0
        asked = False
        dead = False
        while True:
            dead = yield self.item_empty[t % 2], t // 2 - 1
            if dead:
                break
            item = self.items[t] if t < len(self.items) else None
            self.slot[t % 2] = item
            self.item_full[t % 2].arrive()
            if item is None:
                break
            a, b, part = item
            n = max(a, b)
            for k in range(PART):
                if part + k >= n:
                    self.go[t % 2][k].arrive()
            self.next.expect(1)
            self.copies.append(("next", self.next.landed))
            asked = True
            if n:
                dead = yield self.q_empty, n_q - 1
                if dead:
                    break
                self.q_full.expect(1)
                self.copy("q", self.q, n_q, self.q_full)
                n_q += 1
                for i in range(2 * n):
                    dead = yield self.empty[self.ring.stage(use)], use // self.stages - 1
                    if dead:
                        break
                    bar = self.full[self.ring.full(use)]
                    bar.expect(1)
                    self.copy("v" if i & 1 else "k", self.tiles[self.ring.stage(use)], use, bar)
                    if i & 1 and i // 2 >= part:
                        self.go[t % 2][i // 2 - part].arrive()
                    use += 1
            dead = dead or (yield self.next, t)
            if dead:
                break
            asked = False
            t += 1
        for u in range(max(0, use - self.stages), use):
            dead = dead or (yield self.empty[self.ring.stage(u)], u // self.stages, LONG)
        if n_q:
            dead = dead or (yield self.q_empty, n_q - 1, LONG)
        if not dead:
            return
        for u in range(max(0, use - self.stages), use):
            yield (*self.wait_full(u), LANDS)
        if n_q:
            yield self.q_full, n_q - 1, LANDS
        if asked:
            yield self.next, t, LANDS

    def wait_full(self, use):
        return self.full[self.ring.full(use)], self.ring.round(use)

    def drain(self, warp):
        """What a warp that gave up does about its products."""
        self.commit(warp, self.drained[warp])
        yield self.drained[warp], 0, LANDS

    def scores(self):
        use0 = n_q = n_s = t = 0
        while not (yield from self.take(t)):
            item = self.slot[t % 2]
            if item is None:
                return
            n = max(item[:2])
            if n:
                if (yield self.q_full, n_q):
                    break
                n_q += 1
                for j in range(n):
                    use = use0 + 2 * j
                    dead = yield self.wait_full(use)
                    for x in range(2):
                        if j < item[x] and not dead:
                            if n_s:
                                dead = yield self.s_taken, n_s - 1
                            n_s += 1
                            if not dead:
                                self.product("S", [(self.q, n_q - 1), (self.tiles[self.ring.stage(use)], use)])
                                self.commit("S", self.s_full[x])
                    if dead:
                        yield from self.drain("S")
                        return
                    self.commit("S", self.empty[self.ring.stage(use)])
                    if j == n - 1:
                        self.commit("S", self.q_empty)
                use0 += 2 * n
            self.item_empty[t % 2].arrive()
            t += 1
        yield from self.drain("S")

    def sums(self):
        use0, n_p, t = 0, [0, 0], 0
        while not (yield from self.take(t)):
            item = self.slot[t % 2]
            if item is None:
                return
            n = max(item[:2])
            for j in range(n):
                use = use0 + 2 * j + 1
                dead = yield self.wait_full(use)
                if j >= item[2] and not dead:
                    dead = yield self.checked[t % 2][j - item[2]], t // 2
                for x in range(2):
                    if j < item[x] and not dead:
                        dead = yield self.p_full[x], n_p[x]
                        n_p[x] += 1
                        if not dead:
                            self.product("PV", [(self.tiles[self.ring.stage(use)], use)])
                            self.commit("PV", self.pv_done[x])
                if dead:
                    yield from self.drain("PV")
                    return
                self.commit("PV", self.empty[self.ring.stage(use)])
            use0 += 2 * n
            self.item_empty[t % 2].arrive()
            t += 1
        yield from self.drain("PV")

    def check(self):
        use0 = t = 0
        while not (yield from self.take(t)):
            item = self.slot[t % 2]
            if item is None:
                return
            n = max(item[:2])
            for k in range(PART):
                j = item[2] + k
                if j < n:
                    use = use0 + 2 * j + 1
                    if (yield self.go[t % 2][k], t // 2) or (yield self.wait_full(use)):
                        return
                    if self.tiles[self.ring.stage(use)].holds != use:
                        raise Stale("the check of V reads another tile")
                self.checked[t % 2][k].arrive()
            use0 += 2 * n
            self.item_empty[t % 2].arrive()
            t += 1

    def rows(self, x, warp):
        n_s = n_pv = t = 0
        while not (yield from self.take(t)):
            item = self.slot[t % 2]
            if item is None:
                return
            for j in range(item[x]):
                if (yield self.s_full[x], n_s):
                    return
                n_s += 1
                self.s_taken.arrive()
                if j:
                    if (yield self.pv_done[x], n_pv):
                        return
                    n_pv += 1
                self.p_full[x].arrive()
            if item[x]:
                if (yield self.pv_done[x], n_pv):
                    return
                n_pv += 1
            self.rows_done[x].arrive()
            if (yield self.checked[t % 2][PART - 1], t // 2):
                return
            if (yield self.rows_done[x], t, *self.tile_sync):
                return
            self.outputs.append((t, x, warp))
            self.item_empty[t % 2].arrive()
            t += 1

    tile_sync = ()

    # ---- any order
    def run(self):
        roles = {"load": self.load(), "S": self.scores(), "PV": self.sums(), "check": self.check()}
        roles.update({"AB"[x] + str(w): self.rows(x, w) for x in range(2) for w in range(4)})
        kinds = [*roles, "k", "v", "q", "next", "S done", "PV done"]
        pace = {k: 10.0 ** -self.rng.randrange(4) for k in kinds}
        at = {k: next(g) for k, g in roles.items()}
        gave_up = False

        def go_on(k, dead):
            try:
                at[k] = roles[k].send(dead)
            except StopIteration:
                del at[k]
        while True:
            ways, seen = [], set()
            for k, (bar, phase, *_) in at.items():
                if bar.passes(phase):
                    ways.append((k, None))
            for i, (kind, _) in enumerate(self.copies):
                if kind not in seen or self.rng.random() < 0.3:     # (mostly the oldest of a kind)
                    seen.add(kind)
                    ways.append((kind, i))
            ways += [(w + " done", w) for w in self.queue if self.queue[w]]
            out = [k for k, w in at.items() if (len(w) == 2 or w[2] == LONG and not ways) and not w[0].passes(w[1])]   # may run out of time
            if self.gives_up and out and (not ways or self.rng.random() < self.gives_up):
                gave_up = True
                go_on(self.rng.choice(out), True)
                continue
            if not ways:
                break
            k, what = self.rng.choices(ways, [pace[w[0]] for w in ways])[0]
            if k in at:
                go_on(k, False)
            elif isinstance(what, int):
                self.copies.pop(what)[1]()
            else:
                self.queue[what].pop(0)()
            if not at:
                assert not self.copies and not any(self.queue.values()), "the block ends before what it started"
        assert not at and not self.copies, f"nothing goes on: {sorted(at)} wait"
        if not gave_up:
            assert sorted(self.outputs) == [(t, x, w) for t in range(len(self.items)) for x in range(2) for w in range(4)]


class Ring:
    """The header's rule, or one barrier a stage."""

    def __init__(self, stages, lib=None):
        self.stages, self.lib = stages, lib

    def stage(self, use):
        return self.lib.stage(self.stages, use) if self.lib else use % self.stages

    def full(self, use):
        return self.lib.full(self.stages, use) if self.lib else use % self.stages

    def round(self, use):
        """The phase of its barrier that this use is."""
        n = self.lib.fulls(self.stages) if self.lib else self.stages
        if self.lib:
            assert self.lib.full_parity(self.stages, use) == use // n & 1
            assert self.lib.empty_parity(self.stages, use) == use // self.stages & 1
        return use // n


def some_items(rng):
    """Pairs as the kernel makes them: B's tiles are A's or one more, or none (a pair of one tile's tokens)."""
    items = []
    for _ in range(rng.randrange(1, 5)):
        a = rng.choice([0, 1, 2, 3, 4, 6, 9])
        b = rng.choice([0, a, a, a + 1])
        n = max(a, b)
        items.append((a, b, rng.randrange(max(0, n - PART), n + 1)))
    return items


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("ring")
    with open(d / "ring.cpp", "w") as f:
        f.write('#include "tile_ring.h"\n#define BY(name) extern "C" uint32_t name(uint32_t st, uint32_t use) '
                '{ return st == 5 ? mhc::TileRing<5>::name(use) : mhc::TileRing<8>::name(use); }\n'
                'BY(stage) BY(full) BY(full_parity) BY(empty_parity)\n'
                'extern "C" uint32_t fulls(uint32_t st) { return st == 5 ? mhc::TileRing<5>::kFull : mhc::TileRing<8>::kFull; }\n')
    subprocess.run([gxx, "-shared", "-fPIC", "-O1", "-I", os.path.join(ROOT, "manifold_constrained_hyper_mhc_gb300", "csrc"),
                    str(d / "ring.cpp"), "-o", str(d / "ring.so")], check=True)
    return ctypes.CDLL(str(d / "ring.so"))


@pytest.mark.parametrize("stages", [5, 8])   # head_dim 128 and 64
def test_no_wait_passes_early_and_no_product_reads_another_tile(lib, stages):
    ring = Ring(stages, lib)
    for seed in range(800):
        rng = random.Random(seed)
        Model(some_items(rng), stages, ring, rng).run()


def test_a_late_copy_of_v_of_a_pair_with_one_tile(lib):
    """The S of tile j + 1 beside V of tile j - 2 that has not landed: one tile's tokens over many tiles of keys."""
    for seed in range(400):
        rng = random.Random(seed)
        Model([(7, 0, 5), (1, 0, 0), (9, 0, 8)], 5, Ring(5, lib), rng).run()


def test_the_model_sees_one_barrier_for_k_and_v():
    """With one barrier a stage and an odd number of stages such a wait passes early; with an even number it does not."""
    stale = 0
    for seed in range(400):
        rng = random.Random(seed)
        try:
            Model([(7, 0, 5), (1, 0, 0), (9, 0, 8)], 5, Ring(5), rng).run()
        except Stale:
            stale += 1
        rng = random.Random(seed)
        Model([(7, 0, 5), (1, 0, 0), (9, 0, 8)], 8, Ring(8), rng).run()
    assert stale > 0


@pytest.mark.parametrize("stages", [5, 8])
def test_a_wait_that_gives_up_ends_every_role(lib, stages):
    ring = Ring(stages, lib)
    for seed in range(800):
        rng = random.Random(seed)
        Model(some_items(rng), stages, ring, rng, gives_up=rng.choice([0.002, 0.02, 0.2])).run()


def test_the_model_sees_a_barrier_without_a_limit(lib):
    """The warps of a tile at a barrier that none of them leaves before all have come: one that gave up never comes."""
    class Unlimited(Model):
        tile_sync = ("no limit",)
    hung = 0
    for seed in range(400):
        rng = random.Random(seed)
        try:
            Unlimited([(2, 2, 1), (0, 0, 0), (3, 3, 1)], 5, Ring(5, lib), rng, gives_up=0.02).run()
        except AssertionError as e:
            hung += "nothing goes on" in str(e)
    assert hung > 0
