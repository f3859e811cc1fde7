"""The barriers of the shared-prefix decode kernel, as a model on the CPU.

Every role of a CTA (tile producer, the two product issuers, the two softmax
teams, the warp that loads queries) is a generator that yields the barrier
phases it waits for and arrives as the kernel does.  A wait names a parity, as
the hardware's does: it passes when the barrier's current phase has the other
parity, so a wait for a phase that is two away from it blocks for good or
passes too early.  The scheduler picks any role that can go on, at random; no
order may block, and no buffer may be taken before its last reader is done."""
import random

import pytest

SMS = 148


class Cta:
    def __init__(self, case, cta, grid):
        B, Hkv, G, Lp, Lmax, D = case
        R = B * G
        self.key_tiles = -(-Lp // 128)
        row_tiles = -(-R // 128)
        self.F = 1
        for f in (2, 4):
            if R <= 128 // f and Hkv * -(-self.key_tiles // f) >= SMS:
                self.F = f
        self.seg_tiles = -(-self.key_tiles // self.F)
        tiles = Hkv * row_tiles * self.seg_tiles
        own_slots = 0 if Lmax == 0 else 1 if 2 * B * Hkv * Lmax <= Hkv * Lp else 2
        self.stages = (144 * 1024 - own_slots * 8 * 4096) // (128 * D)
        self.psets = 4 // self.F
        each = self.seg_tiles + (4 if tiles > grid else 0)

        def first(i):
            share, more = divmod(Hkv * row_tiles * each, grid)
            p = share * i + min(i, more)
            return p // each * self.seg_tiles + min(p % each, self.seg_tiles)

        assert first(0) == 0 and first(grid) == tiles
        t0, t1 = first(cta), first(cta + 1)
        self.q_stays = t0 < t1 and (t1 - 1) // self.seg_tiles - t0 // self.seg_tiles < 2
        self.segs = []
        while t0 < t1:
            j0 = t0 % self.seg_tiles
            n = min(t1 - t0, self.seg_tiles - j0)
            self.segs.append((j0, n))
            t0 += n
        self.bars = {}
        for name, count, number in (("QFull", 16 if self.q_stays else 1, 2), ("QEmpty", 1, 2), ("SFull", 1, 2),
                                    ("SEmpty", 8, 2), ("PFull", 8, 4), ("PEmpty", 1, 4), ("OFull", 1, 1),
                                    ("OEmpty", 16, 1), ("K", 1, self.stages), ("V", 1, self.stages),
                                    ("Empty", 1, self.stages), ("Team", 2, 1), ("Grid", 2, 1)):
            for i in range(number):
                self.bars[name, i] = [0, count, count]  # phases completed, arrivals missing, arrivals per phase
        self.tile_in = {}              # ring slot -> what was loaded last
        self.s_made = self.pv_done = 0  # tiles of phases A to C with S made; tiles with P.V done

    def folds(self, j):
        return min(self.F, self.key_tiles - j * self.F)

    def arrive(self, name, i=0, n=1):
        b = self.bars[name, i]
        b[1] -= n
        assert b[1] >= 0, f"too many arrivals at {name}{i}"
        if b[1] == 0:
            b[0] += 1
            b[1] = b[2]

    def passes(self, wait):
        name, i, parity = wait
        return self.bars[name, i][0] & 1 != parity & 1

    def producer(self):
        slot, loads = 0, [0] * self.stages
        for phase in range(3):
            for j0, n in self.segs:
                for y in range(2 * n + (4 if phase == 2 else 0)):
                    v = y & 1
                    j = (y >> 1) - 2 * v
                    if j < 0 or j >= n or (v and phase < 2):
                        continue
                    for x in range(self.folds(j0 + j)):
                        yield "Empty", slot, loads[slot] + 1
                        loads[slot] += 1
                        self.tile_in[slot] = ("KV"[v], phase, j0 + j, x)
                        self.arrive("KV"[v], slot)
                        slot = (slot + 1) % self.stages

    def qk_issuer(self):
        slot = sc = nq = 0
        par = [0] * self.stages
        for phase in range(3):
            nq = 0 if self.q_stays else nq
            for j0, n in self.segs:
                yield "QFull", nq & 1, 0 if self.q_stays else nq >> 1
                for e in range(n):
                    yield "SEmpty", sc & 1, (sc >> 1) + 1
                    for x in range(self.folds(j0 + e)):
                        yield "K", slot, par[slot]
                        assert self.tile_in[slot] == ("K", phase, j0 + e, x)
                        par[slot] ^= 1
                        self.arrive("Empty", slot)
                        slot = (slot + 1) % self.stages
                    sc += 1
                    self.s_made = sc
                    self.arrive("SFull", (sc - 1) & 1)
                    if phase == 2 and e >= 2:
                        slot = (slot + self.F) % self.stages
                if phase == 2:
                    for e in range(max(n - 2, 0), n):
                        slot = (slot + self.folds(j0 + e)) % self.stages
                if not self.q_stays:
                    self.arrive("QEmpty", nq & 1)
                nq += 1

    def pv_issuer(self):
        slot = 2 * sum(min((j0 + n) * self.F, self.key_tiles) - j0 * self.F for j0, n in self.segs) % self.stages
        pc = no = 0
        par = [0] * self.stages
        for j0, n in self.segs:
            for e in range(min(n, 2)):
                slot = (slot + self.folds(j0 + e)) % self.stages
            for j in range(n):
                if j + 2 < n:
                    slot = (slot + self.folds(j0 + j + 2)) % self.stages
                p = pc % self.psets
                if j == 0:
                    yield "OEmpty", 0, no + 1
                yield "PFull", p, pc // self.psets
                for x in range(self.folds(j0 + j)):
                    yield "V", slot, par[slot]
                    assert self.tile_in[slot] == ("V", 2, j0 + j, x)
                    par[slot] ^= 1
                    self.arrive("Empty", slot)
                    slot = (slot + 1) % self.stages
                pc += 1
                self.pv_done = pc
                self.arrive("PEmpty", (pc - 1) & 1 if self.psets == 1 else p)
                if j == n - 1:
                    self.arrive("OFull")
            no += 1

    def team(self, team):
        if self.q_stays:
            for i in range(min(len(self.segs), 2)):
                self.arrive("QFull", i, 8)
        sc = pc = teams = 0
        for phase in range(3):
            for no, (j0, n) in enumerate(self.segs):
                if phase:  # the row table
                    self.arrive("Team")
                    yield "Team", 0, teams
                    teams += 1
                for j in range((team - sc) & 1, n, 2):
                    i, pi = sc + j, pc + j
                    yield "SFull", i & 1, i >> 1
                    assert i < self.s_made <= i + 2, "S read before it is made, or after it is gone"
                    if phase == 2:
                        if self.psets == 1:
                            yield "PEmpty", (pi & 1) ^ 1, ((pi + 1) >> 1) - 1
                        else:
                            yield "PEmpty", pi % self.psets, pi // self.psets - 1
                        assert self.pv_done >= pi - self.psets + 1, "P written before its P.V has read it"
                    self.arrive("SEmpty", i & 1, 8)
                    if phase == 2:
                        self.arrive("PFull", pi % self.psets, 8)
                sc += n
                if phase == 2:
                    pc += n
                    yield "OFull", 0, no
                    assert self.pv_done == pc, "O read before it is complete"
                    self.arrive("OEmpty", 0, 8)
                if phase:
                    self.arrive("Team")
                    yield "Team", 0, teams
                    teams += 1
            if phase < 2:
                self.arrive("Grid")
                yield "Grid", 0, phase

    def q_loader(self):
        if not self.q_stays:
            for nq in range(3 * len(self.segs)):
                yield "QEmpty", nq & 1, (nq >> 1) + 1
                self.arrive("QFull", nq & 1)

    def run(self, rng, slow=None):
        """slow: a role that moves only when no other can."""
        roles = {"producer": self.producer(), "qk": self.qk_issuer(), "pv": self.pv_issuer(), "team 0": self.team(0),
                 "team 1": self.team(1), "q": self.q_loader()}
        waits = {}

        def go(k):
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k]

        for k in list(roles):
            go(k)
        while roles:
            able = [k for k in roles if self.passes(waits[k])]
            assert able, f"blocked: {[(k, waits[k]) for k in roles]}"
            go(rng.choice([k for k in able if k != slow] or able))


def _grid(case):
    B, Hkv, G, Lp, Lmax, D = case
    key_tiles, F = -(-Lp // 128), 1
    for f in (2, 4):
        if B * G <= 128 // f and Hkv * -(-key_tiles // f) >= SMS:
            F = f
    return min(SMS, max(Hkv * -(-B * G // 128) * -(-key_tiles // F), B * Hkv * -(-Lmax // 128), 1))


CASES = [  # B, Hkv, G, Lp, Lmax, d
    (4, 20, 1, 37277, 229, 64), (7, 29, 1, 15104, 413, 128), (5, 18, 1, 12841, 805, 128), (1, 26, 1, 37329, 20, 64),
    (2, 11, 3, 21966, 87, 64), (32, 19, 1, 4000, 21, 64), (9, 8, 4, 50000, 333, 128), (64, 8, 4, 8192, 1024, 128),
    (64, 32, 1, 4001, 777, 128), (40, 20, 1, 2100, 17, 64), (400, 100, 1, 100, 3, 64), (129, 8, 4, 250, 5, 128),
    (3, 128, 1, 600, 40, 64), (3, 5, 1, 4100, 0, 64), (2, 16, 1, 4900, 30, 64), (1, 1, 1, 1, 0, 64),
]


@pytest.mark.parametrize("slow", [None, "producer", "qk", "pv", "team 0", "team 1", "q"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}k{}G{}p{}m{}d{}".format(*c))
def test_no_order_blocks(case, slow):
    rng = random.Random(str((case, slow)))
    grid = _grid(case)
    for cta in {0, grid - 1, *(rng.randrange(grid) for _ in range(8))}:
        for _ in range(4):
            Cta(case, cta, grid).run(rng, slow)


def test_drawn_cases():
    rng = random.Random(11)
    for _ in range(300):
        case = (rng.choice([1, 2, 5, 9, 31, 33, 70]), rng.randrange(1, 40), rng.choice([1, 2, 3, 4, 8]),
                int(2 ** rng.uniform(0, 15.5)), rng.choice([0, 9, 100, 800]), rng.choice([64, 128]))
        grid = _grid(case)
        for _ in range(3):
            Cta(case, rng.randrange(grid), grid).run(rng, rng.choice([None, "team 0", "team 1", "pv"]))
