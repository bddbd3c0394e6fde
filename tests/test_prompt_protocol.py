"""The barrier protocol of the prompt attention kernel, model-checked on the CPU under random
interleavings, as tests/test_pipeline_protocol.py does for the GEMMs and with its rules.

Roles: the scheduler (which also looks over V), the TMA producer, one MMA issuer per tile, and W
softmax warps per tile.  Pieces of work are (steps of the first 128 rows, of the second 128, steps
that a mask cuts, whether V of the cut steps holds infinities).  Every buffer carries the tag of what
was last put there: work slots, ring tiles, queries, scores (whose place P takes over), P in its two
parts, and the sums.
"""
import random

import pytest

from test_pipeline_protocol import Barrier, Stale, run

SLOTS, CUTS, W = 4, 3, 2


def prompt_roles(pieces, stages, mistake=None, stores=1):
    B = Barrier
    full = [B(1, f"full{s}") for s in range(stages)]
    empty = [B(1 if mistake == "one tile frees the ring" else 2, f"empty{s}") for s in range(stages)]
    q_full, q_empty = [[B(1, f"{n}{i}") for i in range(2)] for n in ("q_full", "q_empty")]
    s_full, o_full = [[B(1, f"{n}{i}") for i in range(2)] for n in ("s_full", "o_full")]
    p_ready = [[B(W, f"p_ready{i}{k}") for k in range(2)] for i in range(2)]
    o_empty = [B(W, f"o_empty{i}") for i in range(2)]
    turn = [[B(1, f"turn{i}{w}") for w in range(W)] for i in range(2)]
    asked, scan = [[[B(1, f"{n}{s}{c}") for c in range(CUTS)] for s in range(SLOTS)] for n in ("asked", "scan")]
    work_full = [B(1, f"work_full{s}") for s in range(SLOTS)]
    work_empty = [B(3 + 2 * W, f"work_empty{s}") for s in range(SLOTS)]

    def place(i, n):                                       # 0: the first 128 rows, 1: the second
        return i ^ (n & 1)

    def steps_of(n, i):
        return pieces[n][place(i, n)]

    def geometry(n):
        """(steps of the longer tile, first cut step, cut of each place)"""
        a, b, cuts, _ = pieces[n]
        every = max(a, b)
        cut0 = max(0, every - cuts)
        return every, cut0, (cut0, min(cut0 + 1, every))

    def take(n):
        yield "wait", work_full[n % SLOTS], (n // SLOTS) & 1
        yield "read", ("work", n % SLOTS), n

    def scheduler():
        tile = given = 0

        def tell(n):
            if n >= SLOTS and mistake != "work told over work":
                yield "wait", work_empty[n % SLOTS], (n // SLOTS - 1) & 1
            yield "write", ("work", n % SLOTS), n
            yield "arrive", work_full[n % SLOTS]
        for _ in range(2):
            if given <= len(pieces):
                yield from tell(given)                     # the last one says that there is no more
                given += 1
        for n in range(len(pieces)):
            slot, parity = n % SLOTS, (n // SLOTS) & 1
            every, cut0, _ = geometry(n)
            for c in range(CUTS):
                if mistake != "looks before it is asked for":
                    yield "wait", asked[slot][c], parity
                if cut0 + c < every:
                    k = tile + 2 * (cut0 + c) + 1
                    yield "wait", full[k % stages], (k // stages) & 1
                    yield "read", ("ring", k % stages), (n, 2 * (cut0 + c) + 1)
                yield "write", ("dirty", slot, c), n
                yield "arrive", scan[slot][c]
            tile += 2 * every
            if given <= len(pieces):
                yield from tell(given)
                given += 1

    def producer():
        tile = 0
        for n in range(len(pieces)):
            yield from take(n)
            every, cut0, _ = geometry(n)

            def load(k):
                s, turn_of = (tile + k) % stages, (tile + k) // stages
                if turn_of:
                    yield "wait", empty[s], (turn_of - 1) & 1
                yield "write", ("ring", s), None           # from here on the bytes are changing
                yield "arrive", full[s], 1
                yield "copy", full[s], 1, ("ring", s), (n, k)
                if k & 1 and k >> 1 >= cut0:
                    yield "arrive", asked[n % SLOTS][(k >> 1) - cut0]
            if every:
                yield from load(0)
            for i in range(2):
                if n and mistake != "queries over queries":
                    yield "wait", q_empty[i], (n - 1) & 1
                if steps_of(n, i):
                    yield "write", ("q", i), None
                    yield "arrive", q_full[i], 1
                    yield "copy", q_full[i], 1, ("q", i), n
                else:
                    yield "arrive", q_full[i]
            for k in range(1, 2 * every):
                yield from load(k)
            tile += 2 * every
            for c in range(every - cut0, CUTS):
                yield "arrive", asked[n % SLOTS][c]
            yield "arrive", work_empty[n % SLOTS]
        yield from take(len(pieces))

    def issuer(i):
        tile = done = 0
        for n in range(len(pieces)):
            yield from take(n)
            steps, (every, _, cuts) = steps_of(n, i), geometry(n)
            cut, dirty = cuts[place(i, n)], pieces[n][3]
            yield "arrive", work_empty[n % SLOTS]

            def landed(k):
                return "wait", full[(tile + k) % stages], ((tile + k) // stages) & 1

            def scores(j, reads=(), writes=()):
                # with the P V that was issued before it, in one commit
                return ("commit", s_full[i], [*reads, (("ring", (tile + 2 * j) % stages), (n, 2 * j)), (("q", i), n)],
                        [*writes, *((("s", i, w), ("S", n, j)) for w in range(W)),
                         *((("p", i, w, part), None) for w in range(W) for part in range(2))])
            yield "wait", q_full[i], n & 1
            if steps:
                yield landed(0)
                yield scores(0)
            if steps <= 1 or mistake == "queries freed early":
                yield "commit", q_empty[i], []
            if n and mistake != "sums over sums":
                yield "wait", o_empty[i], (n - 1) & 1
            if not steps:
                yield "commit", o_full[i], []
            for j in range(every):
                if j >= steps:
                    for k in (2 * j, 2 * j + 1):
                        if mistake != "passes tiles that have not landed":
                            yield landed(k)
                        yield "commit", empty[(tile + k) % stages], []
                    continue
                yield "commit", empty[(tile + 2 * j) % stages], []
                more = j + 1 < steps
                yield landed(2 * j + 1)
                if more:
                    yield landed(2 * j + 2)
                reads, writes = [], []
                for part in range(2):
                    yield "wait", p_ready[i][part], (done + j) & 1
                    if j >= cut:
                        yield "read", ("skip", i), (n, j, dirty)
                    if j < cut or not dirty:
                        reads += [(("p", i, w, part), (n, j)) for w in range(W)]
                if j < cut or not dirty:
                    reads.append((("ring", (tile + 2 * j + 1) % stages), (n, 2 * j + 1)))
                    if j:
                        reads += [(("o", i, w), (n, j - 1)) for w in range(W)]
                    writes = [(("o", i, w), (n, j)) for w in range(W)]
                if more:
                    yield scores(j + 1, reads, writes)
                    if j + 2 == steps and mistake != "queries freed early":
                        yield "commit", q_empty[i], []
                else:
                    yield "commit", o_full[i], reads, writes
                yield "commit", empty[(tile + 2 * j + 1) % stages], []
            tile += 2 * every
            done += steps
        yield from take(len(pieces))

    def softmax(i, w):
        done = turns = tile = 0
        for n in range(len(pieces)):
            yield from take(n)
            steps, (every, cut0, cuts) = steps_of(n, i), geometry(n)
            cut, dirty, both = cuts[place(i, n)], pieces[n][3], min(pieces[n][:2])
            for j in range(steps):
                yield "wait", s_full[i], (done + j) & 1
                yield "read", ("s", i, w), ("S", n, j)
                if j:
                    yield "read", ("o", i, w), (n, j - 1)  # rescaled here
                before = j - place(i, n)
                if 0 <= before < both:
                    yield "wait", turn[1 - i][w], (turns + before) & 1
                yield "write", ("s", i, w), None           # P takes the place
                yield "write", ("p", i, w, 0), (n, j)
                if j < cut:
                    yield "arrive", p_ready[i][0]
                if j < both:
                    yield "arrive", turn[i][w]
                yield "write", ("p", i, w, 1), (n, j)
                if j >= cut:
                    yield "wait", scan[n % SLOTS][j - cut0], (n // SLOTS) & 1
                    yield "read", ("dirty", n % SLOTS, j - cut0), n
                    yield "write", ("skip", i), (n, j, dirty)
                    if dirty:
                        yield "read", ("ring", (tile + 2 * j + 1) % stages), (n, 2 * j + 1)
                        yield "write", ("o", i, w), (n, j)
                    yield "arrive", p_ready[i][0]
                yield "arrive", p_ready[i][1]
            yield "wait", o_full[i], n & 1
            if steps:
                yield "read", ("o", i, w), (n, steps - 1)
            yield "arrive", o_empty[i]
            for _ in range(stores):
                yield "read", ("work", n % SLOTS), n       # read again for the stores
            tile += 2 * every
            turns += both
            done += steps
            yield "arrive", work_empty[n % SLOTS]
        yield from take(len(pieces))

    return [scheduler(), producer(), issuer(0), issuer(1), *(softmax(i, w) for i in range(2) for w in range(W))]


def random_pieces(rng, count):
    out = []
    for _ in range(count):
        kind = rng.randrange(5)
        first = rng.randrange(1, 6)
        a, b = [(first, first + 1), (first, first), (first, 0), (0, first), (0, 0)][kind]
        out.append((a, b, rng.randrange(1, CUTS + 1), rng.random() < 0.3))
    return out


@pytest.mark.parametrize("stages", [4, 10])
@pytest.mark.parametrize("seed", range(60))
def test_prompt_protocol(seed, stages):
    rng = random.Random(seed)
    pieces = random_pieces(rng, rng.randrange(1, 9))
    for k in range(4):
        run(prompt_roles(pieces, stages, stores=1 if k < 3 else 40), 1000 * seed + k)


@pytest.mark.parametrize("mistake", [
    "one tile frees the ring", "work told over work", "looks before it is asked for", "queries over queries",
    "queries freed early", "sums over sums", "passes tiles that have not landed"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(60):
        rng = random.Random(seed)
        # (work is overtaken only where pieces are short and the stores are long)
        short = mistake == "work told over work"
        pieces = [(1, 1, 1, False)] * 8 if short else random_pieces(rng, 8)
        try:
            run(prompt_roles(pieces, 4, mistake, 100 if short else 1), seed)
        except (Stale, RuntimeError):
            caught += 1
    assert caught
