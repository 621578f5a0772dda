"""More host-side refusals of the full attention and page calls: block tables
that are too short, results that lie over the page state."""
import ctypes

import pytest

from tests.test_serving_calls_cpu import D, call_update, full, state  # noqa: F401 (D is a fixture)


def call_compact(D, st, pools=(), ws=0x900000, ws_bytes=1 << 40, **ptr):
    lib = D.load_library()
    v = dict(table=0x10000, refs=0x20000, remap=None, counts=None)
    v.update(ptr)
    arr = (D.DsaPagePool * max(1, len(pools)))(*[D.DsaPagePool(*x) for x in pools])
    return lib.dsa_pages_compact(ctypes.byref(st), len(pools), arr, v["table"], v["refs"], v["remap"], v["counts"], ws,
                                 ws_bytes, None)


def test_page_calls_refuse_results_over_the_state(D):  # noqa: F811
    import torch
    st = state(D)                                     # a table of 128 bytes, 64 bytes of counts, pools of 16 blocks
    pool = [(0x100000, 256)]
    fine = D.DSA_OK if torch.cuda.is_available() else D.DSA_ERR_NO_DEVICE
    if fine != D.DSA_OK:                              # (nothing may be launched on these addresses)
        assert call_compact(D, st, pool, remap=0x30000, counts=0x30040) == fine
        assert call_compact(D, st, pool, table=0x11000, refs=0x21000, remap=0x20040, counts=0x10080) == fine
        assert call_update(D, st, pool, counts=0x33000) == fine
    bad = D.DSA_ERR_INVALID_ARG
    for out in (dict(), dict(table=0x11000, refs=0x21000)):
        assert call_compact(D, st, pool, remap=0x20000, **out) == bad
        assert call_compact(D, st, pool, remap=0x1ffc4, **out) == bad
        assert call_compact(D, st, pool, remap=0x10070, **out) == bad
        assert call_compact(D, st, pool, counts=0x2003c, **out) == bad
        assert call_compact(D, st, pool, counts=0xfffc, **out) == bad
        assert call_update(D, st, pool, counts=0x2003c, **out) == bad
        assert call_update(D, st, pool, counts=0x10000, **out) == bad
    assert call_compact(D, st, pool, table=0x11000, refs=0x21000, remap=0x21020) == bad
    assert call_compact(D, st, pool, remap=0x30000, counts=0x3003c) == bad
    assert call_compact(D, st, pool, remap=0x100ffc) == bad            # the pool's last bytes
    assert call_update(D, st, pool, counts=0x100000) == bad
    assert call_update(D, st, pool, counts=0x3200c) == bad             # new_len, which the last launch reads
    assert call_update(D, st, pool, parent=0x100100) == bad


def test_a_block_table_needs_a_row_for_every_sequence(D):  # noqa: F811
    import torch
    pages = D.DsaKvPages(128, 10, 4, 0x7000)
    assert D._cache_shapes(full(D), pages) == (1280,)
    for rows in (1, 2, 3):
        pages._table = torch.zeros(rows, 4, dtype=torch.int32)
        if rows < 2:
            with pytest.raises(ValueError, match="rows for 2 sequences"):
                D._cache_shapes(full(D), pages)
        else:
            assert D._cache_shapes(full(D), pages) == (1280,)
