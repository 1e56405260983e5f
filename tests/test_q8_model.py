"""The 8-bit tiles' way through the tensor-core kernel of attention over pages, as a model on the
CPU: the ring of the products with as few stages as it has there, and the landing ring in front of
it with the warps that expand its tiles."""
import random

import numpy as np
import pytest

import q8_ref
import test_paged_models as pm


@pytest.mark.parametrize("stages,own", [(3, False), (4, False), (6, True)])
def test_products_with_a_short_ring(stages, own):
    for seed in range(150):
        pm.run(seed, stages, own)


@pytest.mark.parametrize("raw,stages", [(3, 3), (6, 3), (4, 4), (6, 6), (1, 3)])
def test_landing_ring(raw, stages):
    """Tiles land in any order, four warps expand each of them, two units use and free them."""
    for seed in range(150):
        rnd = random.Random(seed)
        n = rnd.randint(1, 40)
        raw_full, raw_empty = ([pm.Bar(c) for _ in range(raw)] for c in (1, 4))
        kv_full, kv_empty = ([pm.Bar(c) for _ in range(stages)] for c in (4, 2))
        landed, ring, flying = [None] * raw, [[None] * 4 for _ in range(stages)], []

        def load():
            for e in range(n):
                yield from pm.free(raw_empty[e % raw], e // raw)
                flying.append(e)
                yield

        def expand(w):
            for e in range(n):
                yield from pm.full(raw_full[e % raw], e // raw)
                assert landed[e % raw] == e
                yield
                raw_empty[e % raw].arrive()
                yield from pm.free(kv_empty[e % stages], e // stages)
                ring[e % stages][w] = e
                yield
                kv_full[e % stages].arrive()

        def unit():
            for e in range(n):
                yield from pm.full(kv_full[e % stages], e // stages)
                assert ring[e % stages] == [e] * 4
                for _ in range(rnd.randint(0, 5)):
                    yield
                assert ring[e % stages] == [e] * 4
                kv_empty[e % stages].arrive()

        roles = [load(), unit(), unit()] + [expand(w) for w in range(4)]
        weights = [rnd.choice([1, 1, 5, 20]) for _ in roles]
        idle = 0
        while roles:
            if flying and rnd.random() < 0.4:
                e = flying.pop(rnd.randrange(len(flying)))
                landed[e % raw] = e
                raw_full[e % raw].arrive()
            r = rnd.choices(range(len(roles)), weights)[0]
            idle += 1
            assert idle < 200_000, ("no end", seed)
            try:
                next(roles[r])
            except StopIteration:
                del roles[r], weights[r]


def interleave(rnd, roles, events, limit=300_000):
    """Runs coroutines in random turns; events(): what the hardware may do meanwhile."""
    weights = [rnd.choice([1, 1, 5, 20]) for _ in roles]
    idle = 0
    while roles:
        events()
        r = rnd.choices(range(len(roles)), weights)[0]
        idle += 1
        assert idle < limit, "no end"
        try:
            next(roles[r])
        except StopIteration:
            del roles[r], weights[r]


def test_two_stages_of_keys_are_not_enough():
    """A unit's values wait for its next keys, two tiles on, while the other's keys are held."""
    with pytest.raises(AssertionError, match="no end"):
        test_keys_and_values_in_rings_of_their_own(2)


@pytest.mark.parametrize("stages", [3, 4])
def test_keys_and_values_in_rings_of_their_own(stages):
    """Direct keys: a step's tiles in the order of one ring, keys and values each with stages of
    their own; keys are let go with the values of their tile."""
    for seed in range(200):
        rnd = random.Random(seed)
        steps = []
        for _ in range(rnd.randint(1, 6)):
            n, x = rnd.choice([1, 1, 2, 3, 5]), rnd.random()
            steps.append(pm.Step("wide", n) if x < 0.4 else pm.Step("split", n) if x < 0.7 else
                         pm.Step("pair", n, rnd.choice([1, 2, 4])))
        bars = lambda c: [pm.Bar(c) for _ in range(2 * stages)]  # noqa: E731
        raw, full, empty = bars(1), bars(4), bars(2)
        holds, flying, commits = [None] * 2 * stages, [], [[], []]

        def place(s, base, e):
            keys, t = list(s.loads())[e]
            i = base + t
            return (0 if keys else stages) + i % stages, i // stages

        def load():
            base = 0
            for s in steps:
                for e in range(2 * s.n):
                    at, k = place(s, base, e)
                    yield from pm.free(empty[at], k)
                    holds[at] = (base, e)
                    flying.append(raw[at])
                    yield
                base += s.n

        def expand():
            base = 0
            for s in steps:
                for e in range(2 * s.n):
                    at, k = place(s, base, e)
                    yield from pm.full(raw[at], k)
                    assert holds[at] == (base, e)
                    yield
                    full[at].arrive()
                base += s.n

        def products(u):
            base = 0
            for s in steps:
                seen = 0
                split, wide = s.kind == "split", s.kind == "wide"
                n = s.n if split else s.tiles[u]
                first, by = (u, 2) if split else (0, 1)

                def ready(e):
                    nonlocal seen
                    while seen <= e:
                        at, k = place(s, base, seen)
                        yield from pm.full(full[at], k)
                        if not wide and s.owner(seen) != u:
                            empty[at].arrive()
                        seen += 1

                if first < n:
                    yield from ready(s.key(s.tile(u, first)))
                for i in range(first, n, by):
                    t = s.tile(u, i)
                    yield from ready(s.value(t))
                    if i + by < n:
                        yield from ready(s.key(s.tile(u, i + by)))
                    for _ in range(rnd.randint(0, 6)):  # the softmax, which reads the keys' scales
                        yield
                    for e in (s.value(t), s.key(t)):
                        at, _ = place(s, base, e)
                        assert holds[at] == (base, e)
                        commits[u].append(empty[at])
                yield from ready(2 * s.n - 1)
                base += s.n

        def events():
            if flying and rnd.random() < 0.3:
                flying.pop(rnd.randrange(len(flying))).arrive()
            for c in commits:
                if c and rnd.random() < 0.3:
                    c.pop(0).arrive()

        interleave(rnd, [load(), products(0), products(1)] + [expand() for _ in range(4)], events)


@pytest.mark.parametrize("stages,wide", [(2, False), (3, False), (2, True), (3, True)])
def test_pipeline_of_few_rows(stages, wide):
    """The kernel for few rows: load, products (scores a tile ahead), two query warps, expanders and
    softmax warps that meet at every tile.  Wide: weights over their tile of keys, query rows in one
    place."""
    W = 2  # warps of the softmax and of the expanders (the kernel has four)
    for seed in range(250):
        rnd = random.Random(seed)
        items = [rnd.choice([1, 1, 1, 2, 3, 6]) for _ in range(rnd.randint(1, 10))]
        S = stages  # of keys, of values
        two = lambda c, n=2: [pm.Bar(c) for _ in range(n)]  # noqa: E731
        k_full, k_empty, vr_full = two(1, S), two(1 + W, S), two(1, S)
        v_full, v_empty = two(W, S), two(1, S)
        q_full, q_empty, s_full = two(2), two(W if wide else 1 + W), two(1)
        s_empty, o_empty, q_read, held = two(W), two(W), pm.Bar(1), [None]
        p_full, pv_done, vote = pm.Bar(W), pm.Bar(1), pm.Bar(W)
        step_full, step_empty = [pm.Bar(1) for _ in range(4)], [pm.Bar(3 + 2 * W) for _ in range(4)]
        slots, keys, vals, scores = [None] * 4, [None] * S, [None] * S, [None] * 2
        flying, commits = [], []

        def get(j):
            yield from pm.full(step_full[j % 4], j // 4)
            assert slots[j % 4][0] == j
            return slots[j % 4][1]

        def load():
            kp = vp = j = 0
            while (n := (yield from get(j))) is not None:
                for t in range(-1, n):
                    for isk in (True, False):
                        y = t + 1 if isk else t
                        if not 0 <= y < n:
                            continue
                        p = kp if isk else vp
                        yield from pm.free((k_empty if isk else v_empty)[p % S], p // S)
                        (keys if isk else vals)[p % S] = p
                        flying.append((k_full if isk else vr_full)[p % S])
                        kp, vp = kp + isk, vp + (not isk)
                step_empty[j % 4].arrive()
                j += 1

        def convert(i):
            yield from pm.free(q_empty[i & 1], i >> 1)
            if wide:
                yield from pm.free(q_read, i)
                assert held[0] in (None, i - 1, i)
                held[0] = i
            yield
            q_full[i & 1].arrive()

        def query():
            for j in range(len(items) + 1):
                yield from pm.free(step_empty[j % 4], j // 4)
                slots[j % 4] = (j, items[j] if j < len(items) else None)
                yield
                step_full[j % 4].arrive()
                if j:
                    yield from convert(j - 1)

        def second():
            j = 0
            while (yield from get(j)) is not None:
                yield from convert(j)
                step_empty[j % 4].arrive()
                j += 1

        def products():
            jq = tq = iq = jp = tp = ip = 0
            sq = yield from get(0)
            sizes = {0: sq}

            def issue():
                nonlocal jq, tq, iq, sq
                if sq is None:
                    return
                if iq == 0:
                    yield from pm.full(q_full[jq & 1], jq >> 1)
                yield from pm.full(k_full[tq % S], tq // S)
                yield from pm.free(s_empty[tq & 1], tq >> 1)
                assert keys[tq % S] == tq
                scores[tq & 1] = tq
                iq += 1
                assert not wide or held[0] == jq
                commits.extend([s_full[tq & 1]] if wide else [s_full[tq & 1], k_empty[tq % S]])
                if iq == sq:
                    commits.append(q_read if wide else q_empty[jq & 1])
                tq += 1
                if iq == sq:
                    iq, jq = 0, jq + 1
                    sq = sizes[jq] = yield from get(jq)

            yield from issue()
            while tp < tq:
                yield from issue()
                if ip == 0:
                    yield from pm.free(o_empty[jp & 1], jp >> 1)
                yield from pm.full(v_full[tp % S], tp // S)
                yield from pm.full(p_full, tp)
                assert vals[tp % S] == tp and (not wide or keys[tp % S] == ("p", tp))
                commits.extend([pv_done, v_empty[tp % S]] + ([k_empty[tp % S]] if wide else []))
                tp, ip = tp + 1, ip + 1
                if ip == sizes[jp]:
                    step_empty[jp % 4].arrive()
                    ip, jp = 0, jp + 1

        def expand():
            t = j = 0
            while (n := (yield from get(j))) is not None:
                for _ in range(n):
                    yield from pm.full(vr_full[t % S], t // S)
                    assert vals[t % S] == t
                    yield
                    v_full[t % S].arrive()
                    t += 1
                step_empty[j % 4].arrive()
                j += 1

        grown = {}

        def softmax():
            t = nv = j = 0

            def meet():
                nonlocal nv
                vote.arrive()
                yield from pm.full(vote, nv)
                nv += 1

            while (n := (yield from get(j))) is not None:
                yield from pm.full(q_full[j & 1], j >> 1)
                for i in range(n):
                    yield from pm.full(k_full[t % S], t // S)
                    yield from pm.full(s_full[t & 1], t >> 1)
                    assert scores[t & 1] == t and keys[t % S] in (t, ("p", t))
                    yield
                    s_empty[t & 1].arrive()
                    k_empty[t % S].arrive()
                    yield from meet()
                    if grown.setdefault(t, i == 0 or rnd.random() < 0.2):
                        yield from meet()
                        if i:
                            yield from pm.full(pv_done, t - 1)
                    yield from pm.full(vr_full[t % S], t // S)
                    if t:
                        yield from pm.full(pv_done, t - 1)
                    yield
                    if wide:
                        keys[t % S] = ("p", t)
                    p_full.arrive()
                    t += 1
                yield from meet()
                yield from pm.full(pv_done, t - 1)
                o_empty[j & 1].arrive()
                q_empty[j & 1].arrive()
                step_empty[j % 4].arrive()
                j += 1

        def events():
            if flying and rnd.random() < 0.3:
                flying.pop(rnd.randrange(len(flying))).arrive()
            if commits and rnd.random() < 0.4:
                commits.pop(0).arrive()

        interleave(rnd, [load(), query(), second(), products()] + [expand() for _ in range(W)] +
                   [softmax() for _ in range(W)], events)


def test_the_definition_of_a_row():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((200, 32)) * 2.0 ** rng.integers(-140, 120, (200, 1))
    b, s = q8_ref.quantise(y)
    e = s.astype(int) - 127
    got = q8_ref.value(b, s)
    top = np.abs(y).max(1)
    assert (top <= 448 * 2.0 ** e).all()
    assert ((top > 448 * 2.0 ** (e - 1.0)) | (e == q8_ref.LO)).all()
    assert (np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y),
                                          2.0 ** (e[:, None] - 10.0))).all()
    # every finite number is kept as itself
    for k in (q8_ref.LO, -3, 0, 50, q8_ref.HI):
        x = np.concatenate([np.delete(q8_ref.E4M3, [127, 255]), [448.0]])[None] * 2.0 ** k
        b, s = q8_ref.quantise(x)
        assert (q8_ref.value(b, s) == x).all() and s[0] == k + 127
