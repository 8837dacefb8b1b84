"""A beam whose logits are not read, because it has ended or holds nothing, may name any logits row: nothing is flagged,
and an ended beam stays its own candidate."""
import numpy as np
import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn
import test_parity_beam as beam

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row", [-1, 8, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("dead", [-np.inf, np.nan])
def test_rows_of_ended_and_dead_beams(row, dead):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    x = beam._logits(8, 3000, "f32", 30)
    scores = beam._scores(2, 4, 30)
    scores[0, 2] = dead
    finished = np.zeros((2, 4), dtype=np.uint8)
    finished[0, 1] = finished[1, 0] = 1
    good = np.arange(8).reshape(2, 4)
    rows = good.copy()
    rows[0, 1] = rows[0, 2] = rows[1, 0] = row
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = beam._check(x, scores, 6, rows=rows, finished=finished, eos=2, err=err)
    assert int(err.item()) == 0
    same = beam._run(x, scores, 6, rows=good, finished=finished, eos=2)
    for a, b in zip(got, same):
        np.testing.assert_array_equal(a, b)


def test_a_bad_row_of_a_live_beam_is_still_flagged():
    x = beam._logits(8, 3000, "bf16", 31)
    rows = np.array([[0, 8, 2, 3]])
    finished = np.array([[0, 0, 0, 1]], dtype=np.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = beam._run(x, beam._scores(1, 4, 31), 8, rows=rows, finished=finished, eos=2, err=err)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    assert 1 not in got[1][0]
