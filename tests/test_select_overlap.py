"""Outputs of gdn_beam_select over memory that its second launch still reads: refused before any CUDA call, except in
place with one table of the same layout, which gives the same results as separate buffers."""
import ctypes

import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn
import test_beam_abi as abi
import test_parity_beam as beam

FAR = abi.BASE + (40 << 32)


def _valid(K):
    """2 x 4 beams; every buffer in a place of its own."""
    a = abi._select()
    a.K, a.eos_token = K, 2
    for i, f in enumerate(("rows", "finished", "out_finished")):
        setattr(a, f, FAR + (i << 32))
    return a


INPUTS = {"rows": 32, "scores": 32, "finished": 8}
OUTPUTS = {"out_scores": 4, "out_parents": 4, "out_tokens": 4, "out_finished": 1}


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("table", INPUTS)
@pytest.mark.parametrize("K", [3, 8])
def test_an_output_over_a_table_of_another_layout(out, table, K):
    for offset in (0, INPUTS[table] - 4, 4 - 2 * K * OUTPUTS[out]):
        a = _valid(K)
        setattr(a, out, getattr(a, table) + offset)
        assert gdn.lib().gdn_beam_select(ctypes.byref(a), None) == -6, offset


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("table", INPUTS)
def test_an_output_over_part_of_a_table(out, table):
    a = _valid(4)
    setattr(a, out, getattr(a, table) + 4)
    assert gdn.lib().gdn_beam_select(ctypes.byref(a), None) == -6


@pytest.mark.parametrize("out,table", [("out_finished", "rows"), ("out_finished", "scores"), ("out_scores", "finished"),
                                       ("out_parents", "finished"), ("out_tokens", "finished")])
def test_an_output_in_place_of_a_table_of_another_type(out, table):
    a = _valid(4)
    setattr(a, out, getattr(a, table))
    assert gdn.lib().gdn_beam_select(ctypes.byref(a), None) == -6


@pytest.mark.parametrize("out", OUTPUTS)
def test_an_output_in_the_workspace(out):
    a = _valid(4)
    need = gdn.lib().gdn_beam_select_workspace_bytes(a.batch, a.beams, a.vocab, a.K)
    for offset in (0, need - 4):
        setattr(a, out, a.workspace + offset)
        assert gdn.lib().gdn_beam_select(ctypes.byref(a), None) == -6


@pytest.mark.gpu
@pytest.mark.parametrize("batch,beams", [(1, 4), (300, 5)])
def test_in_place(batch, beams):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    V = 4000
    x = beam._logits(batch * beams, V, "bf16", 40)
    scores = torch.from_numpy(beam._scores(batch, beams, 40)).cuda()
    finished = (torch.rand(batch, beams, generator=torch.Generator().manual_seed(40)) < 0.3).to(torch.uint8).cuda()
    rows = torch.randperm(batch * beams, generator=torch.Generator().manual_seed(41)).to(torch.int32).view(batch, beams).cuda()
    ws = gdn.beam_select_workspace(batch, beams, V, beams)
    new = lambda t: torch.full((batch, beams), 7, dtype=t, device="cuda")
    apart = [new(torch.float32), new(torch.int32), new(torch.int32), new(torch.uint8)]
    gdn.gdn_beam_select(x, scores, *apart[:3], rows=rows, finished=finished, eos_token=2, out_finished=apart[3], workspace=ws)
    place = [scores.clone(), rows.clone(), new(torch.int32), finished.clone()]
    gdn.gdn_beam_select(x, place[0], *place[:3], rows=place[1], finished=place[3], eos_token=2, out_finished=place[3], workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(apart, place):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("beams,K", [(1, 4), (4, 2), (3, 9)])
def test_one_entry_in_place(beams, K):
    """A single entry's results may lie over its tables whatever the sizes: all is read before any is written."""
    V = 4000
    x = beam._logits(beams, V, "bf16", 42)
    scores = torch.from_numpy(beam._scores(1, beams, 42)).cuda()
    ws = gdn.beam_select_workspace(1, beams, V, K)
    new = lambda t: torch.full((1, K), 7, dtype=t, device="cuda")
    apart = [new(torch.float32), new(torch.int32), new(torch.int32)]
    gdn.gdn_beam_select(x, scores, *apart, workspace=ws)
    both = torch.zeros(max(beams, K), device="cuda")
    both[:beams] = scores[0]
    place = [both[:K].view(1, K), new(torch.int32), new(torch.int32)]
    gdn.gdn_beam_select(x, both[:beams].view(1, beams), *place, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(apart, place):
        assert torch.equal(a, b)
