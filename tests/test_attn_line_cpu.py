"""The split of mq_attn_decode's work over thread blocks, restated: units of tiles laid on a line
with gaps, equal shares of the line for the blocks, the next tile from any place, and the blocks
that share a unit.  Every tile must be one block's, in order, and the blocks that a unit is counted
over must be those that have tiles of it; planted mistakes must show."""
import random

import pytest


def lay_out(tiles, units, blocks):
    """(gap, steps, spans): spans[i] = (first step, tiles) of unit i on the line."""
    gap = int(sum(tiles) * units >= 4 * blocks)
    at, spans = 0, []
    for n in tiles:
        for _ in range(units if n else 0):
            spans.append((at + gap, n))
            at += n + gap
    return gap, at, spans


def cursor_at(spans, gap, at):
    """The first tile at or after a step: (unit, tile, step)."""
    for u, (first, n) in enumerate(spans):
        if at < first + n:
            tile = max(0, at - first)
            return u, tile, first + tile
    raise AssertionError("a step past the line")


def next_tile(spans, gap, c):
    u, tile, at = c
    tile, at = tile + 1, at + 1
    if tile < spans[u][1]:
        return u, tile, at
    return u + 1, 0, at + gap


def first_and_last(first, n, T, parts, slip=0):
    """Blocks of a unit's first and last tile."""
    return ((first + 1) * parts - 1) // T, ((first + n + slip) * parts - 1) // T


def split(tiles, units, blocks, wrong=None):
    """Checks the split; returns the number of shared units."""
    gap, T, spans = lay_out(tiles, units, blocks)
    if T == 0:
        return 0
    parts = min(blocks, T)
    owner, shared = {}, {}
    for b in range(parts):
        at, end = T * b // parts, T * (b + 1) // parts
        if wrong == "end":
            end -= 1
        c = cursor_at(spans, gap, at)
        split_pieces = []
        while c[2] < end:
            u, tile, at = c
            first, n = spans[u]
            assert at - tile == first
            count = min(end - at, n - tile)
            for i in range(count):
                assert (u, tile + i) not in owner, "a tile of two blocks"
                owner[u, tile + i] = b
            if not (tile == 0 and count == n):
                shared.setdefault(u, []).append(b)
                split_pieces.append(int(tile == 0))  # the piece's place in the workspace
            c = next_tile(spans, gap if wrong != "gap" else 0, (u, tile + count - 1, at + count - 1))
        assert len(split_pieces) <= 2 and len(set(split_pieces)) == len(split_pieces)
    assert len(owner) == sum(n for _, n in spans), "a tile of no block"
    order = [owner[u, i] for u, (_, n) in enumerate(spans) for i in range(n)]
    assert order == sorted(order)
    for u, (first, n) in enumerate(spans):
        b0, b1 = first_and_last(first, n, T, parts, slip=1 if wrong == "last" else 0)
        blocks_of = sorted({owner[u, i] for i in range(n)})
        assert blocks_of == list(range(b0, b1 + 1)), "counted over other blocks than have tiles"
        assert shared.get(u, []) == (blocks_of if len(blocks_of) > 1 else [])
    return len(shared)


def cases(count):
    for seed in range(count):
        r = random.Random(seed)
        top = r.choice([1, 3, 20, 400])
        tiles = [r.choice([0, 1, r.randint(1, top)]) for _ in range(r.randint(1, 60))]
        yield tiles, r.choice([1, 2, 4, 12, 36]), r.choice([1, 7, 152])


def test_every_tile_is_one_blocks():
    shared = sum(split(*c) for c in cases(300))
    assert shared > 1000


@pytest.mark.parametrize("wrong", ["end", "gap", "last"])
def test_planted_mistakes_show(wrong):
    caught = 0
    for c in cases(60):
        try:
            split(*c, wrong=wrong)
        except AssertionError:
            caught += 1
    assert caught > 5
