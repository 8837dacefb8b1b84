"""The binding takes the beam search's tables as [batch, beams] or [batch, K], or flat (or a row or column), and refuses two axes of other
sizes: a transposed table has as many entries, but other ones in each place."""
import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn

B, N, K, V = 3, 4, 2, 50


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


@pytest.mark.parametrize("name,shape", [("rows", (N, B)), ("rows", (B, N + 1)), ("rows", (2, 6)), ("finished", (N, B)),
                                        ("out_parents", (K, B)), ("out_tokens", (K, B)), ("out_finished", (K, B))])
def test_select_refuses_other_tables(monkeypatch, name, shape):
    monkeypatch.setattr(gdn, "_ptr", lambda t, name, dtype=None: None if t is None else t.data_ptr())     # CPU tensors
    t = {"rows": _i(B, N), "finished": torch.zeros(B, N, dtype=torch.uint8), "out_parents": _i(B, K), "out_tokens": _i(B, K),
         "out_finished": torch.zeros(B, K, dtype=torch.uint8)}
    t[name] = torch.zeros(*shape, dtype=t[name].dtype)
    with pytest.raises(ValueError, match=name):
        gdn.gdn_beam_select(torch.zeros(B * N, V), torch.zeros(B, N), torch.zeros(B, K), t["out_parents"], t["out_tokens"],
                            rows=t["rows"], finished=t["finished"], out_finished=t["out_finished"], eos_token=0, prepare=True)


@pytest.mark.parametrize("name", ["parents", "new_slots"])
def test_reorder_refuses_other_tables(monkeypatch, name):
    monkeypatch.setattr(gdn, "_ptr", lambda t, name, dtype=None: None if t is None else t.data_ptr())
    t = {"parents": _i(B, N), "new_slots": _i(B, N)}
    t[name] = _i(N, B)
    with pytest.raises(ValueError, match=name):
        gdn.gdn_beam_reorder([], _i(B, N), t["parents"], t["new_slots"], prepare=True)


def test_flat_tables_are_taken(monkeypatch):
    monkeypatch.setattr(gdn, "_ptr", lambda t, name, dtype=None: None if t is None else t.data_ptr())
    gdn.gdn_beam_select(torch.zeros(B * N, V), torch.zeros(B, N), torch.zeros(B, K), _i(B * K), _i(B * K), rows=_i(B * N),
                        finished=torch.zeros(B * N, dtype=torch.bool), eos_token=0, prepare=True)
    gdn.gdn_beam_reorder([], _i(B, N), _i(B * N), _i(B * N), prepare=True)
    gdn.gdn_beam_reorder([], _i(B, N), _i(B * N, 1), _i(1, B * N), prepare=True)
