"""gdn_beam_reorder refuses, before any CUDA call, a table of new slots that overlaps one that its CTAs are still reading."""
import ctypes

import pytest

import ssm_recurrent_decode_gb300 as gdn
import test_beam_abi as abi


@pytest.mark.parametrize("table", ["slots", "parents"])
@pytest.mark.parametrize("offset", [0, 4, 28, -4, -28])
def test_new_slots_over_a_table_that_is_read(table, offset):
    a, _ = abi._reorder()                        # 2 x 4 beams: tables of 32 bytes
    a.new_slots = getattr(a, table) + offset
    assert gdn.lib().gdn_beam_reorder(ctypes.byref(a), None) == -6


@pytest.mark.parametrize("table", ["slots", "parents"])
@pytest.mark.parametrize("offset", [32, -32])
def test_tables_side_by_side_are_no_overlap(table, offset):
    """Not refused for it: the next check of the host, of a pool, is what answers."""
    a, pools = abi._reorder()
    a.new_slots = getattr(a, table) + offset
    pools[0].base = None
    assert gdn.lib().gdn_beam_reorder(ctypes.byref(a), None) == -1


def test_an_empty_call_overlaps_nothing():
    a, _ = abi._reorder()
    a.batch, a.new_slots = 0, a.parents
    assert gdn.lib().gdn_beam_reorder(ctypes.byref(a), None) == 0
