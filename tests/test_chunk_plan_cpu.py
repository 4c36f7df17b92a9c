"""Chunk attention's bookkeeping re-stated on the CPU: what the plan makes of any
lengths stays within what the host gives, and the ring of images is never
overwritten early, never stuck, and never waits a phase behind."""
import random

SMS, TILE, ROWS, MIN_PIECE, MAX_PIECES, FEW, FINE = 152, 128, 256, 6, 32, 4, 1024


def up(n, d):
    return -(-n // d)


def added(heads):
    return SMS // heads + 1


def host(B, T, heads, total):
    tiles, units = total // TILE + B, T // ROWS + B + 2
    slots = 0 if tiles <= MIN_PIECE else min(units * min(MAX_PIECES, up(tiles, MIN_PIECE)), 2 * added(heads))
    return dict(tiles=tiles, units=units, slots=slots, pieces=units + (added(heads) if slots else 0),
                lo=min(tiles, B * (FINE // TILE)))


def plan(seq, q, T, heads, h):
    """Key tiles of each unit, pieces of each, images and remainders per request."""
    start, lo, n_lo = [0], [], 0
    for s, n in zip(seq, q):
        own = up(s, TILE) if n > 0 and s > 0 else 0
        start.append(start[-1] + own)
        fine = own if s <= FINE else 0
        lo.append(n_lo if fine and n_lo + fine <= h["lo"] else -1)
        n_lo += fine
    start = [min(x, h["tiles"]) for x in start]
    units = []
    for b, (s, n) in enumerate(zip(seq, q)):
        for block in range(up(n, ROWS)):
            end = s - n + min(n, ROWS * (block + 1))
            units.append(up(end, TILE) if end > 0 and start[b + 1] - start[b] >= up(s, TILE) else 0)
    pads = up(T - sum(q), ROWS)
    work = max(1, sum(units) * heads)
    few = (len(units) + pads) * heads * FEW <= SMS
    cuts = [1 if h["slots"] == 0 else
            max(1, min((n * SMS + (0 if few else work - 1)) // work, MAX_PIECES, n // MIN_PIECE)) for n in units]
    return start, lo, units, cuts, pads


def test_plan_stays_in_bounds():
    rng = random.Random(5)
    for _ in range(4000):
        B, heads = rng.randint(1, 12), rng.choice((1, 2, 5, 16, 64, 128))
        seq = [rng.choice((0, rng.randint(0, 300), rng.randint(0, 40000))) for _ in range(B)]
        q = [rng.choice((0, 1, rng.randint(0, 3000))) for _ in range(B)]
        T = sum(q) + rng.choice((0, 7, 700))
        total = sum(seq) if rng.random() < 0.7 else rng.randint(0, sum(seq))
        h = host(B, T, heads, total)
        start, lo, units, cuts, pads = plan(seq, q, T, heads, h)
        assert sum(cuts) + pads <= h["pieces"]
        assert sum(c for c in cuts if c > 1) <= h["slots"]
        assert all(n <= h["tiles"] for n in units)
        for b in range(B):
            if total == sum(seq) and q[b] and seq[b]:  # the host's bound holds: every request's images fit
                assert start[b + 1] - start[b] == up(seq[b], TILE)
                assert (lo[b] >= 0) == (seq[b] <= FINE)
            if lo[b] >= 0:
                assert lo[b] + up(seq[b], TILE) <= h["lo"]
        for n, c in zip(units, cuts):
            edges = [n * i // c for i in range(c + 1)]
            assert edges[-1] == n and (c == 1 or min(b - a for a, b in zip(edges, edges[1:])) >= MIN_PIECE)


SLOTS = 8


def run_ring(fine, n0, n1, rng):
    """Loader, issuer and gate step in random order; P(j) of a group is there once
    its S(j) was issued.  Frees count at issue, which is the earliest."""
    n, images = max(n0, n1), 5 if fine else 3
    per = images + 2
    done = dict(k_free=[0, 0], v_free=[0, 0], k_full=[0, 0], v_full=[0, 0], p=[0, 0])
    held = {}

    def wait(name, o, nth):  # phase `nth` (0, 1, ..) of the barrier: over, and no later one too
        assert done[name][o] <= nth + 1, (name, "two phases behind")
        return done[name][o] > nth

    def put(slot, what):
        old = held.get(slot)
        assert old is None or done[old[0] + "_free"][old[1] & 1] > old[1] >> 1, (slot, what, old)
        held[slot] = what

    def loader():
        for j in range(n):
            o, before = j & 1, (j - 1) & 1
            while j >= 2 and not wait("v_free", o, (j >> 1) - 1):
                yield
            while fine and j >= 1 and not wait("k_free", before, (j - 1) >> 1):
                yield
            for c in range(images):
                put((per * j + c) % SLOTS, ("k", j))
            done["k_full"][o] += 1
            yield
            while j >= 1 and not wait("v_free" if fine else "k_free", before, (j - 1) >> 1):
                yield
            for c in range(2):
                put((per * j + images + c) % SLOTS, ("v", j))
            done["v_full"][o] += 1
            yield

    softmax, gated = [0, 0], [0, 0]

    def gate():
        for j in range(n):
            while not wait("v_full", j & 1, j >> 1):
                yield
            for g, tiles in ((0, n0), (1, n1)):
                if j < tiles:
                    while j > 0 and not wait("p", g, j - 1):
                        yield
                    gated[g] += 1
                    close(g)
                    yield

    def close(g):  # p_full: the softmax's arrivals and the gate's
        done["p"][g] = min(softmax[g], gated[g])

    def issuer():
        for j in range(n + 1):
            for g, tiles in ((0, n0), (1, n1)):
                if 1 <= j <= tiles:
                    while not wait("p", g, j - 1):
                        yield
                    for c in range(2):
                        assert held[(per * (j - 1) + images + c) % SLOTS] == ("v", j - 1)
                if g == 1 and j >= 1:
                    done["v_free"][(j - 1) & 1] += 1
                if j < tiles:
                    if g == 0 or j >= n0:
                        while not wait("k_full", j & 1, j >> 1):
                            yield
                    for c in range(images):
                        assert held[(per * j + c) % SLOTS] == ("k", j)
                    softmax[g] += 1
                    close(g)
                if g == 1 and j < n:
                    done["k_free"][j & 1] += 1
                yield

    roles = [loader(), gate(), issuer()]
    for _ in range(200000):
        if not roles:
            return
        r = rng.choice(roles)
        try:
            next(r)
        except StopIteration:
            roles.remove(r)
    raise AssertionError("stuck")


def test_ring():
    rng = random.Random(6)
    for fine in (False, True):
        for n0 in range(0, 9):
            for n1 in [0] + list(range(max(1, n0), n0 + 3)):
                if max(n0, n1):
                    for _ in range(4):
                        run_ring(fine, n0, n1, rng)
