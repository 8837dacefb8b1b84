"""Gradients of initial states over those of final ones, which one chunk would write while another still reads them, are
refused before any CUDA call."""
import ctypes

import pytest

import ssm_recurrent_decode_gb300 as gdn
import test_scan_abi as abi

ROW = 64 * 16 * 4                               # one state row of test_scan_abi's sizes


@pytest.mark.parametrize("rows", [1, 5])
def test_initial_gradients_over_final_ones(rows):
    for offset in (0, 4, ROW - 4, rows * ROW - 4, -4, 4 - rows * ROW):
        a = abi._valid_grad()
        a.s.num_states = rows
        a.dh0 = a.dh_last + offset
        assert gdn.lib().mamba_selective_scan_backward(ctypes.byref(a), None) == -6, offset


def test_buffers_side_by_side_are_no_overlap():
    """Not refused for it: the next check of the host, of the workspace, is what answers."""
    for offset in (ROW, -ROW):
        a = abi._valid_grad()
        a.dh0, a.s.workspace = a.dh_last + offset, None
        assert gdn.lib().mamba_selective_scan_backward(ctypes.byref(a), None) == -1
