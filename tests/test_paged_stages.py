"""CPU check of the stages of K in the row-tile kernel's units of one row tile.

There every other key tile is one product warp's and the rest the other's. A
warp waits for tile u at barrier u % barriers by the parity of its round, u //
barriers: that says "landed" too early while the round before has not landed
yet. A warp knows that of its own tiles only, so the tile that had the barrier
before has to be one of its own, or of an earlier piece. All orders in which
copies may land and warps may move are walked here."""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_tiled_gb300", "csrc",
                      "fa_paged_tile.cu")


def early(stages, barriers, pieces):
    """Whether some order of events lets a wait pass before its tile landed."""
    tiles, n = [[], []], 0                      # (tile, tiles of the pieces before) of each warp
    for length in pieces:
        for t in range(length):
            tiles[t & 1].append((n + t, n))
        n += length
    # requested: a count, in order; landed and done: sets of tiles; at: each warp's place; passed: its wait is over
    start = (0, frozenset(), frozenset(), (0, 0), (False, False))
    seen, todo = {start}, [start]

    def go(*state):
        if state not in seen:
            seen.add(state)
            todo.append(state)

    while todo:
        requested, landed, done, at, passed = todo.pop()
        if requested < n and (requested < stages or requested - stages in done):
            go(requested + 1, landed, done, at, passed)
        for u in range(requested):
            # a stage's copies follow one another; others may overtake
            if u not in landed:
                go(requested, landed | {u}, done, at, passed)
        for w in range(2):
            if at[w] == len(tiles[w]):
                continue
            u, before = tiles[w][at[w]]
            if passed[w]:                       # the products, and with them the stage's release
                go(requested, landed, done | {u}, tuple(x + (i == w) for i, x in enumerate(at)),
                   tuple(x and i != w for i, x in enumerate(passed)))
                continue
            if len([x for x in done if x < before]) < before:
                continue                        # a piece's Q comes once both warps are through with the piece before
            rounds = len([x for x in landed if x % barriers == u % barriers])
            if rounds % 2 != (u // barriers) & 1:
                if u not in landed:
                    return True
                go(requested, landed, done, at, tuple(x or i == w for i, x in enumerate(passed)))
    return False


PIECES = [(9,), (3, 6), (1, 1, 5), (2, 1, 4), (4, 3)]


def one_row_tile_stages():
    with open(SOURCE) as f:
        text = f.read()
    stages = re.search(r"int KS = D == 128 \? \(ONE \? (\d+) : \d+\) : (\d+);", text).groups()
    assert "int KB = ONE && KS % 2 ? 2 * KS : KS;" in text
    return [(int(x), int(x) * (1 + int(x) % 2)) for x in stages]


@pytest.mark.parametrize("pieces", PIECES)
def test_no_wait_for_k_passes_early(pieces):
    for stages, barriers in one_row_tile_stages():
        assert not early(stages, barriers, pieces), (stages, barriers)


def test_the_walk_finds_early_waits():
    """With an odd number of barriers the tile before at a barrier is the other warp's."""
    assert early(3, 3, (9,)) and early(5, 5, (9,))
    assert not early(2, 2, (9,)) and not early(4, 4, (9,)) and not early(3, 6, (9,))
