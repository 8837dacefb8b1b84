"""CPU checks of the beam search operators: their references by hand, refusals before any CUDA call, sizes."""
import ctypes

import numpy as np
import pytest

import beam_reference as ref
import ssm_recurrent_decode_gb300 as gdn

BASE = 1 << 40


def test_reference_selects_by_hand():
    logits = np.log(np.array([[0.5, 0.25, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4]]) + 0.0, where=np.array([[1, 1, 1, 0], [1] * 4], bool),
                    out=np.full((2, 4), -np.inf))
    s, p, t, _ = ref.select(logits, np.array([[0.0, np.log(0.9)]]), 4)
    np.testing.assert_array_equal(p[0], [0, 1, 1, 0])
    np.testing.assert_array_equal(t[0], [0, 3, 2, 1])
    np.testing.assert_allclose(np.exp(s[0]), [0.5, 0.36, 0.27, 0.25], rtol=1e-12)
    s, p, t, _ = ref.select(logits, np.array([[0.0, -0.1]]), 2, finished=np.array([[0, 1]]), eos=3)
    np.testing.assert_array_equal(p[0], [1, 0])
    np.testing.assert_array_equal(t[0], [3, 0])


def test_reference_reorders_by_hand():
    new, copies = ref.reorder(np.array([[10, 11, 12, 13]]), np.array([[2, 2, 0, 2]]))
    np.testing.assert_array_equal(new, [[12, 11, 10, 13]])
    assert copies == [(12, 11), (12, 13)]
    new, copies = ref.reorder(np.array([[5, 6, 7]]), np.array([[-1, 1, 3]]))
    np.testing.assert_array_equal(new, [[5, 6, 7]])
    assert copies == []


def _select():
    a = gdn.BeamSelectArgs()
    a.batch, a.beams, a.vocab, a.K, a.logits_dtype, a.num_rows = 2, 4, 1000, 8, gdn.GDN_BF16, 8
    for i, f in enumerate(("logits", "scores", "out_scores", "out_parents", "out_tokens", "workspace")):
        setattr(a, f, BASE + (i << 32))
    a.row_stride, a.workspace_bytes = 1000, 1 << 20
    return a


REFUSED_SELECT = [
    ("no logits", lambda a: setattr(a, "logits", None), -1),
    ("no scores", lambda a: setattr(a, "scores", None), -1),
    ("no output", lambda a: setattr(a, "out_tokens", None), -1),
    ("no workspace", lambda a: setattr(a, "workspace", None), -1),
    ("no beam", lambda a: setattr(a, "beams", 0), -2),
    ("too many beams", lambda a: setattr(a, "beams", 33), -2),
    ("no token", lambda a: setattr(a, "vocab", 0), -2),
    ("K of zero", lambda a: setattr(a, "K", 0), -2),
    ("K too large", lambda a: setattr(a, "K", 65), -2),
    ("negative batch", lambda a: setattr(a, "batch", -1), -2),
    ("row stride below the row", lambda a: setattr(a, "row_stride", 999), -2),
    ("too few rows", lambda a: setattr(a, "num_rows", 7), -2),
    ("workspace too small", lambda a: setattr(a, "workspace_bytes", 64), -2),
    ("logits type", lambda a: setattr(a, "logits_dtype", 3), -3),
    ("logits not on an element", lambda a: setattr(a, "logits", BASE + 1), -4),
    ("workspace not on 16 bytes", lambda a: setattr(a, "workspace", BASE + 8), -4),
    ("end token outside the vocabulary", lambda a: (setattr(a, "finished", BASE), setattr(a, "eos_token", 1000)), -6),
    ("no end token", lambda a: (setattr(a, "out_finished", BASE), setattr(a, "eos_token", -1)), -6),
]


@pytest.mark.parametrize("name,mutate,code", REFUSED_SELECT, ids=[r[0] for r in REFUSED_SELECT])
def test_select_refuses_on_the_host(name, mutate, code):
    a = _select()
    mutate(a)
    assert gdn.lib().gdn_beam_select(ctypes.byref(a), None) == code


def _reorder():
    a = gdn.BeamReorderArgs()
    a.batch, a.beams, a.num_slots, a.num_pools = 2, 4, 8, 2
    pools = (gdn.BeamPool * 2)()
    for i, p in enumerate(pools):
        p.base, p.slot_stride, p.slot_bytes = BASE + (i << 34), 4096, 4000
    a.pools = pools
    a.slots, a.parents, a.new_slots = BASE + (9 << 34), BASE + (10 << 34), BASE + (11 << 34)
    return a, pools


REFUSED_REORDER = [
    ("no slots", lambda a, p: setattr(a, "slots", None), -1),
    ("no pool table", lambda a, p: setattr(a, "pools", None), -1),
    ("a pool without memory", lambda a, p: setattr(p[1], "base", None), -1),
    ("too many beams", lambda a, p: setattr(a, "beams", 33), -2),
    ("no slot", lambda a, p: setattr(a, "num_slots", 0), -2),
    ("too many pools", lambda a, p: setattr(a, "num_pools", 129), -2),
    ("negative batch", lambda a, p: setattr(a, "batch", -1), -2),
    ("slots that overlap", lambda a, p: setattr(p[0], "slot_stride", 3999), -2),
    ("slots not on an element", lambda a, p: setattr(a, "slots", BASE + 2), -4),
    ("new slots over the old", lambda a, p: setattr(a, "new_slots", a.slots), -6),
]


@pytest.mark.parametrize("name,mutate,code", REFUSED_REORDER, ids=[r[0] for r in REFUSED_REORDER])
def test_reorder_refuses_on_the_host(name, mutate, code):
    a, pools = _reorder()
    mutate(a, pools)
    assert gdn.lib().gdn_beam_reorder(ctypes.byref(a), None) == code


def test_nothing_to_do_and_sizes():
    L = gdn.lib()
    assert L.gdn_beam_select(None, None) == -1 and L.gdn_beam_reorder(None, None) == -1
    a = _select()
    a.batch = 0
    assert L.gdn_beam_select(ctypes.byref(a), None) == 0
    b, _ = _reorder()
    b.batch = 0
    assert L.gdn_beam_reorder(ctypes.byref(b), None) == 0
    assert L.gdn_abi_struct_size(8) == ctypes.sizeof(gdn.BeamSelectArgs)
    assert L.gdn_abi_struct_size(10) == ctypes.sizeof(gdn.BeamReorderArgs)
    f = L.gdn_beam_select_workspace_bytes
    assert f(1, 4, 32000, 4) >= 4 * 4 * 8
    assert f(1, 33, 100, 4) == 0 and f(1, 1, 0, 1) == 0 and f(1, 1, 1, 65) == 0


def test_binding_checks():
    torch = pytest.importorskip("torch")
    z, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        gdn.gdn_beam_select(z(4, 10), z(1, 4), z(1, 4), i(1, 4), i(1, 4))
    with pytest.raises(ValueError, match="inner stride"):
        gdn.gdn_beam_select(z(10, 4).t(), z(1, 4), z(1, 4), i(1, 4), i(1, 4))
    with pytest.raises(ValueError, match="same number of slots"):
        gdn.gdn_beam_reorder([z(0), z(3, 4)], i(1, 2), i(1, 2), i(1, 2))
