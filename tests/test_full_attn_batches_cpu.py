"""The batches of the full attention tests give the thread blocks the work
that they are meant to, by a restatement of the schedule."""
import pytest

from tests import _full_attn_batches as F


@pytest.mark.parametrize("name", list(F.MIXED))
def test_mixed_batches_go_from_narrow_to_wide_items(name):
    to_rows, _ = F.changes(F.segments(**F.MIXED[name]))
    # an odd number of tiles from three up: the last tile is not the slot's that is done first
    assert any(n >= 3 and n % 2 for n in to_rows)


@pytest.mark.parametrize("name", list(F.NO_KEY))
def test_padded_batches_have_runs_of_items_without_a_key(name):
    slot = F.constants()["kSlotRows"]
    blocks = F.segments(**F.NO_KEY[name])
    runs = [sum(n == 0 and (rows > slot or "5_tokens" in name) for rows, n, _ in b) for b in blocks]
    assert max(runs) >= (2 if name == "padded_batch" else 25)
    assert any(n for b in blocks for _, n, _ in b)
