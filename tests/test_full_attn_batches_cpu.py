"""The batches of the full attention tests give the thread blocks the work
that they are meant to, by a restatement of the schedule."""
import pytest

from tests import _full_attn_batches as F


@pytest.mark.parametrize("name", list(F.MIXED))
def test_mixed_batches_go_from_narrow_to_wide_items(name):
    to_rows, _ = F.changes(F.segments(**F.MIXED[name]))
    # an odd number of tiles from three up: the last tile is not the slot's that is done first
    assert any(n >= 3 and n % 2 for n in to_rows)


@pytest.mark.parametrize("name", list(F.ONE_TILE))
def test_one_tile_batches_go_from_narrow_items_of_one_tile_to_wide_ones(name):
    to_rows, _ = F.changes(F.segments(**F.ONE_TILE[name]))
    assert to_rows.count(1) >= 10


def test_padded_batches_have_runs_of_items_without_a_key():
    """Several in one block, of more than 128 rows, before items with keys and behind them; spread over
    the blocks, however many there are."""
    slot = F.constants()["kSlotRows"]
    before = after = longest = 0
    for name, c in F.NO_KEY.items():
        blocks = F.segments(**c)
        empty = [sum(n == 0 for _, n, _ in b) for b in blocks]
        assert any(n for b in blocks for _, n, _ in b) and any(empty)
        assert max(empty) <= 20, name
        for b in blocks:
            run = 0
            for (r0, n0, _), (r1, n1, _) in zip(b, b[1:]):
                run = run + 1 if n0 == n1 == 0 and r0 > slot and r1 > slot else 0
                longest = max(longest, run + 1)
                before += n0 == 0 and n1 > 0 and r0 > slot
                after += n0 > 0 and n1 == 0 and r1 > slot
    assert longest >= 5 and before and after


def test_loop_batches_cover_the_main_loop():
    """Segments of several tiles, odd and even, in items of up to 128 rows and in wider ones; blocks of
    several segments; changes between the two kinds, after odd and even numbers of tiles; parts and whole
    items."""
    slot = F.constants()["kSlotRows"]
    blocks = {name: F.segments(**c) for name, c in F.LOOPS.items()}
    for name, b in blocks.items():
        assert sum(n for x in b for _, n, _ in x) >= 3 * F.SMS, name
        assert sum(n >= 3 for x in b for _, n, _ in x) >= F.SMS // 2, name
    segs = [s for b in blocks.values() for x in b for s in x]
    for narrow in (True, False):
        here = [(n, whole) for rows, n, whole in segs if (rows <= slot) == narrow]
        assert {n % 2 for n, _ in here if n >= 3} == {0, 1}
        assert {whole for n, whole in here if n >= 3} == {True, False}
    to_rows = [n for b in blocks.values() for n in F.changes(b)[0]]
    to_keys = [n for b in blocks.values() for n in F.changes(b)[1]]
    assert {n % 2 for n in to_rows} == {n % 2 for n in to_keys} == {0, 1}
    assert any(len(x) >= 3 for x in blocks["many_short"])
