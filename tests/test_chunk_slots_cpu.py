"""Chunk attention's slots for the pieces of cut units, as the library's own
workspace size has them, against what the plan makes of any lengths."""
import random

from tests.test_chunk_plan_cpu import FINE, MAX_PIECES, MIN_PIECE, ROWS, SMS, TILE, added, plan, up
import mla_decode_context_gb300 as dcp

IMAGE, SLOT, PIECE = 16384, ROWS * 129 * 4, 64


def round256(n):
    return up(n, 256) * 256


def host(B, T, heads, total):
    """Tiles, units and pieces as the host counts them; slots out of the library."""
    tiles, units = total // TILE + B, T // ROWS + B + 2
    lo = min(tiles, B * (FINE // TILE))
    image = tiles * (4 * IMAGE + 16) + lo * 2 * IMAGE
    assert image * heads <= 4 << 30  # (more heads would not be in one pass)
    at = round256((3 * (B + 1) + 1) * 4)
    at = round256(at + (units + added(1)) * PIECE)
    at = round256(at + tiles * 16) + tiles * IMAGE
    rest = dcp.dcp_chunk_attention_workspace_size(B, T, heads, total) - at - round256(image * heads)
    slots, over = divmod(rest, SLOT * heads)
    assert over == 0 and slots >= 0
    return dict(tiles=tiles, units=units, slots=slots, pieces=units + (added(heads) if slots else 0), lo=lo)


def test_pieces_fit_the_librarys_slots():
    rng = random.Random(7)
    cut = 0
    for _ in range(4000):
        B, heads = rng.randint(1, 12), rng.choice((1, 2, 5, 16, 64, 128))
        top = min(40000, (4 << 30) // (heads * 66000 * B) * TILE - 2 * TILE)
        seq = [rng.choice((0, rng.randint(0, 300), rng.randint(1300, 1700), rng.randint(0, top))) for _ in range(B)]
        if heads * (sum(seq) // TILE + 9 * B) * 100000 > 4 << 30:
            continue
        q = [rng.choice((0, 1, rng.randint(0, 3000))) for _ in range(B)]
        T = sum(q) + rng.choice((1, 7, 700))
        h = host(B, T, heads, sum(seq))
        _, _, units, cuts, pads = plan(seq, q, T, heads, h)
        assert sum(cuts) + pads <= h["pieces"]
        assert sum(c for c in cuts if c > 1) <= h["slots"]
        # none where no unit is long enough to be cut into two pieces, and as many as any
        # lengths of that sum can use otherwise
        longest = h["tiles"] // MIN_PIECE
        assert (h["slots"] == 0) == (longest < 2)
        if h["slots"]:
            assert h["slots"] == min(h["units"] * min(MAX_PIECES, up(h["tiles"], MIN_PIECE)), 2 * added(heads))
            assert all(c <= max(1, n // MIN_PIECE) for n, c in zip(units, cuts))
        cut += any(c > 1 for c in cuts)
    assert cut > 200
    assert added(1) == SMS + 1
