"""The roles of the 8-bit decode's scan (copies of keys and of values, score and
value products, softmax, value sums) as coroutines over barriers that know the
parity of their phase only, run over random schedules: what every role reads is
checked to be what it is meant to read, and nothing gets stuck.  A model of
decode8.cu's order of waits and arrivals, not of its arithmetic; mistakes put
into it are found."""
import random

import pytest

SOFTMAX, VALUES = 8, 4     # warps


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase, self.bytes = count, count, 0, 0

    def arrive(self):
        assert self.left > 0, "too many arrivals"
        self.left -= 1
        self._turn()

    def expect(self):
        self.bytes += 1
        self.arrive()

    def land(self):
        assert self.bytes > 0, "a copy that nobody expects"
        self.bytes -= 1
        self._turn()

    def _turn(self):
        if self.left == 0 and self.bytes == 0:
            self.phase, self.left = self.phase + 1, self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class Named:
    """bar.sync among four warps."""

    def __init__(self):
        self.here, self.turn = 0, 0

    def sync(self):
        turn = self.turn
        self.here += 1
        if self.here == 4:
            self.here, self.turn = 0, turn + 1
        yield self, turn

    def done(self, turn):
        return self.turn != turn


def run(pieces, chunks, rings, seed, mistake=""):
    """One CTA: `pieces` holds the tiles of each piece, `chunks` the boxes of a tile, `rings` the slots of the keys' and
    the values' ring.  AssertionError: a role met something else than it meant to."""
    rng = random.Random(seed)
    tiles = [(p, t == n - 1) for p, n in enumerate(pieces) for t in range(n)]
    apart = [rng.random() < 0.5 for _ in tiles]          # tiles whose scales take the softmax's second turn
    one_ring = mistake == "one ring"
    slots = sum(rings)
    full, empty = [Barrier(1) for _ in range(slots)], [Barrier(1) for _ in range(slots)]
    ifull, iempty = [Barrier(1) for _ in "ab"], [Barrier(1 + SOFTMAX) for _ in "ab"]
    sfull, sempty = [Barrier(1) for _ in "ab"], [Barrier(SOFTMAX) for _ in "ab"]
    pfull, pv = [Barrier(SOFTMAX) for _ in "ab"], [Barrier(1) for _ in "ab"]
    oempty = [Barrier(VALUES) for _ in range(chunks)]
    named = [Named(), Named()]
    ring, image, scores, products = [None] * slots, [None] * 2, [None] * 2, [None] * chunks
    probs = [[None] * SOFTMAX for _ in "ab"]
    facs = 2 if mistake == "two factors" else 4
    factors = [None] * facs
    maxima = {(a, h, w): None for a in (0, 1) for h in (0, 1) for w in range(4)}
    tops = {(h, w): None for h in (0, 1) for w in range(4)}
    in_flight, queue = [], {"scores": [], "values": []}   # copies land in any order, products of a warp in theirs

    def place(values, i, j):
        """(slot, phase, copies before it) of box j of tile i."""
        if one_ring:
            at, n, first = i * 2 * chunks + values * chunks + j, slots, 0
        else:
            at, n, first = i * chunks + j, rings[values], values * rings[0]
        return first + at % n, at // n & 1, at // n

    def copies(values):
        piece, current, first = 0, None, True

        def operands(p):
            nonlocal piece
            if piece >= 2:
                yield iempty[piece & 1], (piece >> 1) - 1 & 1
            k, piece = piece & 1, piece + 1
            ifull[k].expect()

            def land():
                image[k] = p
                ifull[k].land()
            in_flight.append(land)

        for i, (p, _) in enumerate(tiles):
            if p != current:
                current = p
                if not values and not first:
                    yield from operands(p)
            for j in range(chunks):
                slot, phase, turn = place(values, i, j)
                if first and not values and turn:       # the ring is full: the first scores are waited for
                    first = False
                    yield from operands(p)
                if turn:
                    yield empty[slot], phase ^ 1
                full[slot].expect()

                def land(slot=slot, tag=(values, i, j)):
                    ring[slot] = tag
                    full[slot].land()
                in_flight.append(land)
                yield None
            if first and not values:
                yield from operands(p)
            first = False

    def score_products():
        piece, current = -1, None
        for i, (p, last) in enumerate(tiles):
            if p != current:
                current, piece = p, piece + 1
                yield ifull[piece & 1], piece >> 1 & 1
            a, k = i & 1, piece & 1
            if i >= 2 and mistake != "scores not waited for":
                yield sempty[a], (i >> 1) - 1 & 1
            for j in range(chunks):
                slot, phase, _ = place(False, i, j)
                yield full[slot], phase
                assert ring[slot] == (False, i, j)

                def product(slot=slot, tag=(False, i, j), p=p, k=k, a=a):
                    assert ring[slot] == tag and image[k] == p
                    scores[a] = "half done"
                queue["scores"] += [product, empty[slot].arrive]

            def commit(a=a, i=i):
                scores[a] = i
                sfull[a].arrive()
            queue["scores"].append(commit)
            if last:
                queue["scores"].append(iempty[k].arrive)
            yield None

    def value_products():
        for i in range(len(tiles)):
            yield pfull[i & 1], i >> 1 & 1
            for j in range(chunks):
                slot, phase, _ = place(True, i, j)
                yield full[slot], phase
                if i > 0 and mistake != "products not waited for":
                    yield oempty[j], i - 1 & 1
                assert ring[slot] == (True, i, j)

                def product(slot=slot, i=i, j=j):
                    assert ring[slot] == (True, i, j) and probs[i & 1] == [i] * SOFTMAX
                    products[j] = i
                queue["values"] += [product, empty[slot].arrive]
            queue["values"].append(pv[i & 1].arrive)

    def softmax(w):
        piece, current, half, quad = -1, None, w >> 2, w & 3
        for i, (p, last) in enumerate(tiles):
            if p != current:
                current, piece = p, piece + 1
                yield ifull[piece & 1], piece >> 1 & 1
                assert image[piece & 1] == p
                iempty[piece & 1].arrive()
            yield sfull[i & 1], i >> 1 & 1
            assert scores[i & 1] == i
            yield None
            assert scores[i & 1] == i
            sempty[i & 1].arrive()
            a = 0 if mistake == "one buffer of maxima" else i & 1
            maxima[a, half, quad] = i
            yield from named[half].sync()
            for q in range(4):
                assert maxima[a, half, q] == i
                yield None
            if apart[i]:
                tops[half, quad] = i
                yield from named[half].sync()
                for q in range(4):
                    assert tops[half, q] == i
                    yield None
            if i > 1 and mistake != "probabilities not waited for":
                yield pv[i & 1], (i >> 1) - 1 & 1
            probs[i & 1][w] = i
            if w == 0:
                factors[i % facs] = i
            yield None
            pfull[i & 1].arrive()
            if last:
                yield from named[half].sync()
                yield from named[half].sync()

    def value_sums():
        for i in range(len(tiles)):
            yield pv[i & 1], i >> 1 & 1
            assert factors[i % facs] == i
            for j in range(chunks):
                assert products[j] == i
                yield None
                assert products[j] == i
                oempty[j].arrive()
                yield None
                assert factors[i % facs] == i

    roles = [copies(0), copies(1), score_products(), value_products()]
    roles += [softmax(w) for w in range(SOFTMAX)] + [value_sums() for _ in range(VALUES)]
    waits, alive = [None] * len(roles), list(range(len(roles)))
    pace = [rng.choice([1, 1, 1, 0.05]) for _ in roles]     # some are slow
    idle = 0
    while alive or in_flight or queue["scores"] or queue["values"]:
        x, moved = rng.random(), True
        if x < 0.25 and in_flight:
            in_flight.pop(rng.randrange(len(in_flight)))()
        elif x < 0.4 and queue["scores"]:
            queue["scores"].pop(0)()
        elif x < 0.55 and queue["values"]:
            queue["values"].pop(0)()
        else:
            moved = False
            if alive:
                r = rng.choice(alive)
                if rng.random() <= pace[r] and (waits[r] is None or waits[r][0].done(waits[r][1])):
                    moved = True
                    try:
                        waits[r] = next(roles[r])
                    except StopIteration:
                        alive.remove(r)
        idle = 0 if moved else idle + 1
        assert idle < 20000, "stuck"


def case(seed):
    rng = random.Random(seed)
    return [rng.randint(1, 4) for _ in range(rng.randint(1, 5))], rng.randint(1, 6), (rng.randint(1, 7), rng.randint(1, 7))


@pytest.mark.parametrize("block", range(8))
def test_every_role_reads_what_it_is_meant_to(block):
    for seed in range(40 * block, 40 * block + 40):
        pieces, chunks, rings = case(seed)
        run(pieces, chunks, rings, seed)


@pytest.mark.parametrize("mistake", ["one ring", "two factors", "scores not waited for", "products not waited for",
                                     "probabilities not waited for", "one buffer of maxima"])
def test_mistakes_are_found(mistake):
    for seed in range(400):
        pieces, chunks, rings = case(seed)
        try:
            run([n + 2 for n in pieces], chunks, rings, seed, mistake)
        except AssertionError:
            return
    pytest.fail("no schedule shows it")
