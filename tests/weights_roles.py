"""A model of how fa_kv_weights_tile_kernel gives out its units and of what its roles wait for, on the CPU.

The units of a launch, their row blocks and the two ways in which clusters get them are found as the kernel finds
them.  Every role of every CTA of a cluster is a generator that yields conditions in the order of the kernel's
waits, with mbarriers as counts.  A role goes on only when its condition holds, so a set of waits that can never
be met shows as a run that comes to rest too early, whatever the timing on a GPU would be.
"""
from __future__ import annotations

TILE, UNITS, RING = 128, 8, {64: 8, 128: 6}

# B, H, Hk, T, d, page, lens, new, left: more units to a cluster than are described ahead, and behind one with row blocks
# a run without any for some CTA.  Ordered by cost in the third and fourth; in the last two the second CTA of a cluster
# has none in a sequence of few new tokens.
CASES = [
    (2, 8, 8, 64, 64, 128, [32768, 32500], None, 128),
    (4, 8, 8, 300, 128, 64, [10000, 12000, 9000, 10240], None, 500),
    (2, 16, 2, 640, 64, 256, [20000, 30000], [640, 637], 200),
    (2, 16, 2, 640, 128, 64, [20000, 30016], [639, 640], 0),
    (2, 4, 4, 2048, 64, 64, [2300, 40000], [2048, 100], -1),
    (2, 4, 4, 2048, 128, 64, [3000, 40960], [2048, 1], -1),
]


def sequences(lens, new, T, left, decay):
    """(len, fresh, lo, hi) of each sequence: the keys whose weights change."""
    out = []
    for n, m in zip(lens, new):
        n, m = max(0, n), max(0, min(m, T))
        hi = n if m else 0
        lo = max(0, n - m - left) if left >= 0 and decay == 1 else 0
        out.append((n, m, min(lo, hi), hi))
    return out


def key_tokens(key, n, m, left, right):
    base = n - m
    a = max(0, key - base - right) if right >= 0 else 0
    b = min(m, key - base + left + 1) if left >= 0 else m
    return min(a, m), max(b, 0)


def plan(B, H, Hk, T, lens, new, left, right, decay, capacity, sms):
    """(units of each cluster in its order, CTAs of a cluster, whether by cost): a unit is the row blocks it has."""
    G, rows = H // Hk, H // Hk * T
    seqs = sequences(lens, new, T, left, decay)
    blocks_most = -(-rows // 128)
    most = B * Hk * -(-capacity // (2 * TILE))
    ranks = 2 if blocks_most >= 16 else 1
    if blocks_most >= 4 and 4 * most <= sms:
        ranks = 4
    elif blocks_most >= 2 and 2 * most <= sms:
        ranks = 2
    clusters = min(sms // ranks, most)
    uneven = blocks_most >= 20 * ranks and clusters <= 96
    line, weight = [], 0
    for n, m, lo, hi in seqs:
        pairs = (-(-hi // TILE) - lo // TILE + 1) // 2 if hi > lo else 0
        weight += pairs * (-(-m // 128) * G - 20 * ranks)
        unit = []
        for i in range(pairs):
            k0 = (lo // TILE + 2 * i) * TILE
            ta, tb = key_tokens(k0, n, m, left, right)[0], key_tokens(min(k0 + 2 * TILE, hi) - 1, n, m, left, right)[1]
            unit.append(0 if tb <= ta else -(-(tb - ta) // 128) * G if T >= 128 else blocks_most)
        line += unit * Hk
    uneven = uneven and weight >= 0
    mine = [[] for _ in range(clusters)]
    if not uneven:
        for i, n in enumerate(line):
            mine[i % clusters].append(n)
    else:
        load = [0] * clusters
        for i, n in enumerate(line):
            c = i if i < clusters else min(range(clusters), key=lambda x: (load[x], x))
            load[c] += min(-(-n // ranks), 1 << 14) + 2
            mine[c].append(n)
    return mine, ranks, uneven


class _Cta:
    def __init__(self, ring):
        self.told = 0                       # units described
        self.read = dict.fromkeys("PMSWE", 0)  # units read by producer, MMA, side, writer, compute warps
        self.free = ring                    # slots of the ring
        self.landed = 0                     # tiles that landed
        self.scores = [0, 0]                # blocks whose products are in S buffer 0 / 1
        self.side = [0, 0]                  # and whose LSE and tokens are beside it
        self.used = [0, 0]                  # blocks of it that the compute warps are done with
        self.sums = [0, 0]                  # units that group 0 / 1 has handed over
        self.taken = 0                      # units that the writer has taken
        self.sent = 0                       # units whose sums went to the first CTA


def run(units, ranks, depth, ring, side_ahead):
    """Whether a cluster with these units (blocks of each) comes to its end; side_ahead: the side warp looks for its
    next block, over units without any, before it hands over the one it holds."""
    ctas = [_Cta(ring) for _ in range(ranks)]
    last = len(units)  # the description that says there is none

    def read(c, who):
        i = c.read[who]
        yield lambda: c.told > i
        c.read[who] += 1

    def mine(r, i):
        return max(0, -(-(units[i] - r) // ranks))

    def producer(c, r):
        yield from read(c, "P")
        for i in range(last):
            n = mine(r, i)
            looked = False
            if n:
                yield lambda: c.free >= 2
                c.free -= 2
                c.landed += 2
            wait = min(8, max(n - 1, 0)) if depth == 3 else 0
            for j in range(n):
                if j == wait:
                    yield from read(c, "P")
                    looked = True
                yield lambda: c.free >= 1
                c.free -= 1
                c.landed += 1
            if not looked:
                yield from read(c, "P")

    def mma(c, r):
        block = taken = 0
        for i in range(last):
            yield from read(c, "M")
            n = mine(r, i)
            taken += 2 if n else 0
            for _ in range(n):
                taken += 1
                yield lambda: c.landed >= taken
                buf, before = block & 1, block >> 1
                yield lambda: c.used[buf] >= before
                c.scores[buf] += 1
                c.free += 1
                block += 1
            c.free += 2 if n else 0
        yield from read(c, "M")

    def hand_over(c, block):
        yield lambda: c.used[block & 1] >= block >> 1
        c.side[block & 1] += 1

    def side(c, r):
        block, held = 0, []
        for i in range(last):
            yield from read(c, "S")
            for _ in range(mine(r, i)):
                for b in held:  # found by now: the block after it
                    yield from hand_over(c, b)
                held = [block] if side_ahead else []
                if not side_ahead:
                    yield from hand_over(c, block)
                block += 1
        yield from read(c, "S")
        for b in held:
            yield from hand_over(c, b)

    def compute(c, r):
        block = 0
        for i in range(last):
            yield from read(c, "E")
            for _ in range(mine(r, i)):
                buf, n = block & 1, block >> 1
                yield lambda: c.scores[buf] > n and c.side[buf] > n
                c.used[buf] += 1
                block += 1
            yield lambda: c.taken >= i - 1
            c.sums[i & 1] += 1
        yield from read(c, "E")

    def writer(c, r):
        def tell():
            if c.told <= last:
                yield lambda: min(c.read.values()) >= c.told - UNITS + 1
                c.told += 1

        for _ in range(depth):
            yield from tell()
        for i in range(last):
            yield from read(c, "W")
            yield lambda: c.sums[i & 1] > i >> 1
            c.sent += 1
            if r == 0:
                yield lambda: all(o.sent > i for o in ctas)
            else:
                yield lambda: ctas[0].taken > i
            c.taken += 1
            yield from tell()
        yield from read(c, "W")

    live = [(role(c, r), None) for r, c in enumerate(ctas) for role in (producer, mma, side, compute, writer)]
    while live:
        moved, progress = [], False
        for g, cond in live:
            while cond is None or cond():
                progress = True
                try:
                    cond = next(g)
                except StopIteration:
                    g = None
                    break
            if g is not None:
                moved.append((g, cond))
        if not progress:
            return False
        live = moved
    return True


def stalls(side_ahead, B, H, Hk, T, d, lens, new, left, right, decay, capacity, sms=152):
    """(clusters that come to rest too early, CTAs of a cluster, by cost, most units of a cluster); new None: T each."""
    new = [T] * B if new is None else new
    mine, ranks, uneven = plan(B, H, Hk, T, lens, new, left, right, decay, capacity, sms)
    depth = 3 if uneven else UNITS - 1
    bad = sum(not run(u, ranks, depth, RING[d], side_ahead) for u in mine)
    return bad, ranks, uneven, max(map(len, mine))
