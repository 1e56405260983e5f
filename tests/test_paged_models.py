"""Models of paged attention's tensor-core kernel, run on the CPU.

The pipeline: its roles as coroutines that are interleaved at random, every wait checked the way
the hardware decides it.  A barrier is waited for by the parity of its phase, so that a waiter that
is two phases off would pass or block wrongly: each look at a barrier asserts that it is not.  The
ring's stages remember which entry they hold, and each use asserts that it is the one meant.

The line: items of random batches cut into stretches, every tile worked on exactly once, and the
joined parts those that were left."""
import random
from collections import deque

import pytest

CTAS, TILE, ROWS, UNIT_ROWS = 152, 128, 256, 128
AHEAD, WARPS = 4, 2  # steps put down ahead; softmax warps of a unit (the kernel has four)


# ------------------------------------------------------------------------------ the pipeline

class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1


def full(bar, k):
    """Until the k-th phase is complete (parity k & 1)."""
    while True:
        assert k <= bar.phase <= k + 1
        if bar.phase == k + 1:
            return
        yield


def free(bar, k):
    """Until the k-th use may begin: the phase before it is complete (parity (k & 1) ^ 1)."""
    while True:
        assert k - 1 <= bar.phase <= k
        if bar.phase == k:
            return
        yield


class Step:
    """wide: n tiles for both units; split: n tiles taken in turn; pair: n[u] tiles for each."""

    def __init__(self, kind, n0, n1=0):
        self.kind, self.tiles = kind, (n0, n1 if kind == "pair" else n0)
        self.n = n0 + n1
        self.turns = 2 * min(n0, n1) if kind == "pair" else self.n
        self.longer = int(n1 > n0)

    def tile(self, u, i):
        if self.kind != "pair":
            return i
        return 2 * i + u if 2 * i < self.turns else self.turns // 2 + i

    def key(self, t):
        return 2 * t if self.kind == "wide" else max(2 * t - 1, 0)

    def value(self, t):
        return 2 * t + 1 if self.kind == "wide" else min(2 * t + 2, 2 * self.n - 1)

    def owner(self, e):
        t = self.n - 1 if e == 2 * self.n - 1 else (e + 1) // 2 if e & 1 else max(e // 2 - 1, 0)
        if self.kind == "split":
            return t & 1
        return t & 1 if t < self.turns else self.longer

    def loads(self):
        """(keys or values, tile) as the load warp brings them."""
        for t in range(-1, self.n):
            for keys in (True, False) if self.kind != "wide" else (False, True):
                y = t + 1 if keys else t
                if 0 <= y < self.n:
                    yield keys, y


def test_entries_are_where_the_products_look_for_them():
    for a in range(1, 9):
        for s in [Step("wide", a), Step("split", a)] + [Step("pair", a, b) for b in range(1, 9)]:
            loads = list(s.loads())
            assert len(loads) == 2 * s.n
            for u in range(2):
                mine = range(s.tiles[u]) if s.kind != "split" else range(u, s.n, 2)
                for t in (s.tile(u, i) for i in mine):
                    assert loads[s.key(t)] == (True, t) and loads[s.value(t)] == (False, t)
                    if s.kind != "wide":
                        assert s.owner(s.key(t)) == s.owner(s.value(t)) == u


def run(seed, stages, own):
    """One CTA's life.  own: weights in columns of their own (head dims of at most 64)."""
    rnd = random.Random(seed)

    def make():
        n, x = rnd.choice([1, 1, 1, 2, 3, 4, 7]), rnd.random()
        return (Step("wide", n) if x < 0.3 else Step("split", n) if x < 0.55 else
                Step("pair", n, rnd.choice([1, 1, 2, 3, 4, 7])))

    steps = [make() for _ in range(rnd.randint(1, 12))]
    two = lambda c: [Bar(c), Bar(c)]  # noqa: E731
    kv_full, kv_empty = [Bar(1) for _ in range(stages)], [Bar(2) for _ in range(stages)]
    q_full, q_empty, s_full, o_full, oh_full, turn = two(1), two(2), two(1), two(1), two(1), two(1)
    s_empty, p_full, ph_full, join = two(WARPS), two(WARPS), two(WARPS), Bar(2 * WARPS)
    step_full = [Bar(1) for _ in range(AHEAD)]
    step_empty = [Bar(3 + 2 * WARPS) for _ in range(AHEAD)]
    slots, holds = [None] * AHEAD, [None] * stages
    flying, commits = [], [deque(), deque()]  # copies in any order; a unit's commits in theirs

    def get(j):
        yield from full(step_full[j % AHEAD], j // AHEAD)
        assert slots[j % AHEAD][0] == j
        return slots[j % AHEAD][1]

    def load():
        pos = j = 0
        while (s := (yield from get(j))) is not None:
            for _ in s.loads():
                yield from free(kv_empty[pos % stages], pos // stages)
                holds[pos % stages] = pos
                flying.append(kv_full[pos % stages])
                pos += 1
                yield
            step_empty[j % AHEAD].arrive()
            j += 1

    def query():
        used = [0, 0]
        for j in range(len(steps) + 1):
            yield from free(step_empty[j % AHEAD], j // AHEAD)
            slots[j % AHEAD] = (j, steps[j] if j < len(steps) else None)
            yield
            step_full[j % AHEAD].arrive()
            for t in range(0 if j == 0 else 1 if steps[j - 1].kind == "split" else 2):
                yield from free(q_empty[t], used[t])
                used[t] += 1
                yield
                flying.append(q_full[t])

    def products(u):
        pos = seen = handed = items = wides = turns = scores = j = 0
        commit = commits[u].append
        while (s := (yield from get(j))) is not None:
            split, wide = s.kind == "split", s.kind == "wide"
            tile, n = (0, s.n) if split else (u, s.tiles[u])
            first, by = (u, 2) if split else (0, 1)

            def ready(at):
                nonlocal seen
                while seen <= at:
                    yield from full(kv_full[seen % stages], seen // stages)
                    if not wide and s.owner(seen - pos) != u:
                        kv_empty[seen % stages].arrive()
                    seen += 1

            def use(at):
                assert holds[at % stages] == at
                return kv_empty[at % stages]

            def scores_free():
                nonlocal scores
                if own:
                    yield from free(s_empty[u], scores)
                scores += 1

            def let_query_go():
                for _ in range(1 + (tile == 1)):
                    commit(q_empty[tile])

            yield from full(q_full[0], items)
            if tile:
                q_empty[0].arrive()
                yield from full(q_full[1], wides)
            items, wides = items + 1, wides + (not split)
            if first < n:
                k = pos + s.key(s.tile(u, first))
                yield from ready(k)
                yield from scores_free()
                commit(s_full[u])
                commit(use(k))
                if first + by >= n:
                    let_query_go()
            else:
                q_empty[tile].arrive()
            for i in range(first, n, by):
                more = i + by < n
                v = pos + s.value(s.tile(u, i))
                k = pos + s.key(s.tile(u, i + by)) if more else None
                if own:
                    if more:
                        yield from ready(k)
                        yield from scores_free()
                        commit(s_full[u])
                        commit(use(k))
                        if i + 2 * by >= n:
                            let_query_go()
                    yield from ready(v)
                    yield from full(p_full[u], handed)
                    handed += 1
                    commit(o_full[u])
                    commit(use(v))
                else:
                    yield from ready(v)
                    if more:
                        yield from ready(k)
                    yield from full(ph_full[u], handed)
                    if wide:
                        yield from (full if u else free)(turn[u], turns)
                        turns += 1
                    commit(oh_full[u])
                    yield
                    yield from full(p_full[u], handed)
                    handed += 1
                    if wide:
                        turn[1 - u].arrive()
                    commit(s_full[u] if more else o_full[u])
                    commit(use(v))
                    if more:
                        commit(use(k))
                        if i + 2 * by >= n:
                            let_query_go()
            yield from ready(pos + 2 * s.n - 1)
            pos += 2 * s.n
            step_empty[j % AHEAD].arrive()
            j += 1

    def softmax(u):
        tiles = outs = pos = joins = j = 0
        while (s := (yield from get(j))) is not None:
            split = s.kind == "split"
            n = s.n if split else s.tiles[u]
            mine = 0
            for i in range(u if split else 0, n, 2 if split else 1):
                yield from full(s_full[u], tiles)
                tiles += 1
                halves = False
                if own:  # scores read, and the last weights' product done: in either order
                    for what in rnd.sample([0, 1], 2):
                        if what:
                            s_empty[u].arrive()
                        else:
                            yield from free(o_full[u], outs)
                        yield
                elif rnd.random() < 0.4:  # the lower half handed over ahead
                    ph_full[u].arrive()
                    halves = True
                    yield
                    if rnd.random() < 0.3:  # ... and O scaled before the upper one
                        yield from full(oh_full[u], tiles - 1)
                if rnd.random() < 0.5:  # values cleared
                    at = pos + s.value(s.tile(u, i))
                    yield from full(kv_full[at % stages], at // stages)
                    assert holds[at % stages] == at
                for _ in range(rnd.randint(0, 4)):
                    yield
                if not own and not halves:
                    ph_full[u].arrive()
                p_full[u].arrive()
                mine += 1
                outs += own
            if mine:
                outs += not own
                yield from free(o_full[u], outs)
            for _ in range(2 * split):
                join.arrive()
                yield from full(join, joins)
                joins += 1
            pos += 2 * s.n
            step_empty[j % AHEAD].arrive()
            j += 1

    roles = [load(), query(), products(0), products(1)] + [
        softmax(u) for u in (0, 1) for _ in range(WARPS)]
    weights = [rnd.choice([1, 1, 5, 20]) for _ in roles]
    idle = 0
    while roles:
        if flying and rnd.random() < 0.3:
            flying.pop(rnd.randrange(len(flying))).arrive()
        for c in commits:
            if c and rnd.random() < 0.3:
                c.popleft().arrive()
        r = rnd.choices(range(len(roles)), weights)[0]
        idle += 1
        assert idle < 400_000, ("no end", seed, [(s.kind, s.tiles) for s in steps])
        try:
            next(roles[r])
        except StopIteration:
            del roles[r], weights[r]
    assert not flying


@pytest.mark.parametrize("stages,own", [(5, False), (8, True)])
def test_pipeline(stages, own):
    for seed in range(250):
        run(seed, stages, own)


# ---------------------------------------------------------------------------------- the line

def geometry(new, kv, G, window, sinks, rt, wide_extra):
    """Tiles of a sequence's row tile, and the units that lie before them in the line."""
    row0 = rt * ROWS
    rows, pos0 = min(ROWS, new * G - row0), kv - new
    t0, t1 = row0 // G, (row0 + rows - 1) // G
    hi = max(min(kv, pos0 + t1 + 1), 0)
    lo = min(max(0, max(pos0 + t0, 0) - window + 1) if window else 0, hi)
    first = lo // TILE
    head = min((min(sinks if window else 0, lo) + TILE - 1) // TILE, first)
    return max(head + (hi + TILE - 1) // TILE - first, 1), wide_extra if rows > UNIT_ROWS else 2


def stretch(total, c):
    return total // CTAS * c + min(c, total % CTAS)


def test_line():
    for seed in range(300):
        rnd = random.Random(seed)
        Hkv, G = rnd.choice([1, 2, 3, 8]), rnd.choice([1, 2, 4, 5, 8])
        window, sinks = rnd.choice([0, 0, rnd.randint(1, 500)]), rnd.choice([0, 4, 300])
        extra = rnd.choice([2, 3])
        items = []  # (tiles, units before them)
        for _ in range(rnd.randint(1, 30)):
            new, past = rnd.choice([0, 1, 1, 1, 2, rnd.randint(1, 700)]), rnd.randint(0, 3000)
            kv = new + past if rnd.random() < 0.9 else max(0, new - past)
            items += [geometry(new, kv, G, window, sinks, rt, extra)
                      for _ in range(Hkv) for rt in range(-(-new * G // ROWS))]
        starts, total = [], 0
        for tiles, before in items:
            starts.append(total)
            total += tiles + before
        done = [[0] * tiles for tiles, _ in items]
        parts, headers = {}, {}  # slot 2 c (an item's middle or end), 2 c + 1 (its start)
        for c in range(CTAS):
            a, end = stretch(total, c), stretch(total, c + 1)
            k = max((i for i, s in enumerate(starts) if s <= a), default=None)
            while k is not None and a < end:
                tiles, before = items[k]
                last = min(starts[k] + tiles + before, end)
                v0 = max(a - starts[k] - before, 0)
                v1 = max(last - starts[k] - before, 0)
                if v1 <= v0:
                    break  # the next CTA takes the item whole
                for v in range(v0, v1):
                    done[k][v] += 1
                if v0 > 0 or v1 < tiles:
                    slot = 2 * c + (v0 == 0)
                    assert slot not in parts
                    parts[slot] = (k, v1 - v0)
                    if v0 == 0:
                        headers[c] = (k, end - v1)
                a, k = last, k + 1
        assert all(x == 1 for d in done for x in d)
        joined = set()
        for c, (k, at) in headers.items():
            tiles = items[k][0]
            assert at == starts[k] + items[k][1]
            seen = 0
            for p in range(c, CTAS):
                first, last = stretch(total, p) - at, min(stretch(total, p + 1) - at, tiles)
                if last > max(first, 0):
                    slot = 2 * p + (p == c)
                    assert parts[slot][0] == k
                    joined.add(slot)
                    seen += parts[slot][1]
            assert seen == tiles
        assert joined == set(parts)
