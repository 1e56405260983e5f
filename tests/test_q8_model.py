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
