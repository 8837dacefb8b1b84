"""Host-side checks of linear attention and rotary positions: argument structs and refusals that reach no launch
(the device addresses are aligned and never dereferenced)."""
import ctypes
import math

import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn

NULL, SHAPE, DTYPE, ALIGN, ARG = -1, -2, -3, -4, -6
HUGE = 1 << 40


def at(i):
    return HUGE + (i << 32)


def linear(**kw):
    a = gdn.LinearArgs()
    a.T, a.S, a.H, a.HV, a.K, a.V, a.in_dtype, a.out_dtype = 96, 2, 2, 4, 64, 48, 1, 1
    for i, (n, heads, dim) in enumerate((("q", 2, 64), ("k", 2, 64), ("v", 4, 48), ("o", 4, 48))):
        setattr(a, n, at(i))
        setattr(a, n + "_stride", heads * dim)
        setattr(a, n + "_head_stride", dim)
    a.g, a.g_stride, a.num_states = at(5), 4, 2
    a.workspace, a.workspace_bytes = at(6), 1 << 31
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def call(a):
    return gdn.lib().gdn_linear_attention(ctypes.byref(a), None)


@pytest.mark.parametrize("change,status", [
    ({"q": None}, NULL), ({"k": None}, NULL), ({"v": None}, NULL), ({"g": None}, NULL), ({"o": None}, NULL),
    ({"T": -1}, SHAPE), ({"S": 0}, SHAPE), ({"S": 5}, SHAPE), ({"H": 3}, SHAPE), ({"HV": 0}, SHAPE), ({"K": 48}, SHAPE), ({"K": 256}, SHAPE),
    ({"V": 0}, SHAPE), ({"V": 129}, SHAPE), ({"in_dtype": 2}, DTYPE), ({"out_dtype": 7}, DTYPE),
    ({"q": at(0) + 1}, ALIGN), ({"o": at(3) + 1}, ALIGN), ({"g": at(5) + 2}, ALIGN), ({"final_state": at(7) + 4}, ALIGN),
    ({"initial_state": at(7) + 8}, ALIGN), ({"q_stride": -64}, SHAPE), ({"v_head_stride": -1}, SHAPE),
    ({"o_stride": 100}, SHAPE), ({"o_head_stride": 40}, SHAPE), ({"final_state": at(7), "num_states": 1}, SHAPE),
    ({"final_state": at(7), "num_states": 0}, SHAPE),
])
def test_refusals(change, status):
    assert call(linear(**change)) == status


def test_workspace_is_checked_where_one_is_needed():
    n = gdn.lib().gdn_linear_workspace_bytes(4096, 1, 2, 4, 64, 48, 1, 1, 0)
    assert n > 0
    big = {"T": 4096, "S": 1}
    assert call(linear(**big, workspace=None)) == NULL
    assert call(linear(**big, workspace_bytes=n - 1)) == SHAPE
    assert call(linear(**big, workspace=at(6) + 8, workspace_bytes=n)) == ALIGN
    for bad in ((-1, 1, 2, 4, 64, 48), (5, 2, 2, 4, 64, 48), (8, 1, 3, 4, 64, 48), (8, 1, 2, 4, 63, 48), (8, 1, 2, 4, 64, 0)):
        assert gdn.lib().gdn_linear_workspace_bytes(*bad, 1, 1, 0) == 0


def test_nothing_to_do():
    assert call(linear(T=0, workspace=None)) == 0
    assert gdn.lib().gdn_linear_attention(None, None) == NULL


def grad(**kw):
    a = gdn.LinearGradArgs()
    a.s = linear()
    for i, (n, heads, dim) in enumerate((("dq", 2, 64), ("dk", 2, 64), ("dv", 4, 48), ("d_o", 4, 48))):
        setattr(a, n, at(10 + i))
        s = "do" if n == "d_o" else n
        setattr(a, s + "_stride", heads * dim)
        setattr(a, s + "_head_stride", dim)
    a.dg, a.dg_stride = at(15), 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({"d_o": None}, NULL), ({"dq": at(10) + 1}, ALIGN), ({"dg": at(15) + 1}, ALIGN), ({"dq_stride": 64}, SHAPE),
    ({"dv_head_stride": 47}, SHAPE), ({"dg_stride": 3}, SHAPE), ({"do_stride": -1}, SHAPE),
    ({"d_initial_state": at(17), "d_final_state": at(17)}, ARG), ({"d_initial_state": at(17) + 16, "d_final_state": at(17)}, ARG),
    ({"d_initial_state": at(17) + 8}, ALIGN), ({"s": linear(T=95)}, SHAPE), ({"s": linear(workspace=None)}, NULL),
    ({"s": linear(initial_state=at(17)), "d_initial_state": at(17)}, ARG),
])
def test_gradient_refusals(change, status):
    assert gdn.lib().gdn_linear_attention_backward(ctypes.byref(grad(**change)), None) == status


def step(**kw):
    a = gdn.LinearStepArgs()
    a.B, a.H, a.HV, a.K, a.V, a.num_slots, a.in_dtype, a.out_dtype, a.state_dtype = 3, 2, 4, 64, 48, 5, 1, 1, 0
    for i, (n, heads, dim) in enumerate((("q", 2, 64), ("k", 2, 64), ("v", 4, 48))):
        setattr(a, n, at(i))
        setattr(a, n + "_stride", heads * dim)
        setattr(a, n + "_head_stride", dim)
    a.g, a.state, a.out = at(4), at(5), at(6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({"B": -1}, SHAPE), ({"HV": 3}, SHAPE), ({"K": 24}, SHAPE), ({"V": 0}, SHAPE), ({"V": 1025}, SHAPE), ({"num_slots": 0}, SHAPE),
    ({"num_slots": 2}, SHAPE), ({"in_dtype": 3}, DTYPE), ({"state_dtype": 2}, DTYPE), ({"q": None}, NULL), ({"g": None}, NULL),
    ({"state": None}, NULL), ({"state": at(5) + 8}, ALIGN), ({"v": at(2) + 1}, ALIGN), ({"rotary_dim": 3}, SHAPE),
    ({"rotary_dim": 66}, SHAPE), ({"rotary_dim": 32}, NULL), ({"k_stride": -2}, SHAPE),
    ({"rotary_dim": 32, "positions": at(8), "frequencies": at(9) + 4}, ALIGN),
])
def test_step_refusals(change, status):
    assert gdn.lib().gdn_linear_attention_step(ctypes.byref(step(**change)), None, -1, None) == status


def rotary(**kw):
    a = gdn.RotaryArgs()
    a.T, a.H, a.HK, a.D, a.rotary_dim, a.dtype = 7, 3, 2, 64, 32, 1
    for i, (n, heads) in enumerate((("q", 3), ("q_out", 3), ("k", 2), ("k_out", 2))):
        setattr(a, n, at(i))
        setattr(a, n + "_stride", heads * 64)
        setattr(a, n + "_head_stride", 64)
    a.positions, a.frequencies = at(5), at(6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, SHAPE), ({"H": 0}, SHAPE), ({"HK": -1}, SHAPE), ({"D": 1}, SHAPE), ({"D": 2048}, SHAPE), ({"rotary_dim": 31}, SHAPE),
    ({"rotary_dim": 0}, SHAPE), ({"rotary_dim": 66}, SHAPE), ({"dtype": 2}, DTYPE), ({"positions": None}, NULL),
    ({"frequencies": None}, NULL), ({"k_out": None}, NULL), ({"q": None}, NULL), ({"q": at(0) + 1}, ALIGN),
    ({"frequencies": at(6) + 4}, ALIGN), ({"q_out_stride": 64}, SHAPE), ({"q_out_head_stride": 32}, SHAPE), ({"k_stride": -1}, SHAPE),
    ({"q_out": at(0), "q_out_stride": 256}, ARG),
])
def test_rotary_refusals(change, status):
    assert gdn.lib().gdn_rotary(ctypes.byref(rotary(**change)), None) == status


def test_struct_sizes():
    for which, cls in ((12, gdn.LinearArgs), (13, gdn.LinearGradArgs), (14, gdn.LinearStepArgs), (15, gdn.RotaryArgs)):
        assert gdn.lib().gdn_abi_struct_size(which) == ctypes.sizeof(cls)


def test_the_binding_has_no_cpu_path():
    t = torch.zeros(4, 2, 16)
    with pytest.raises(TypeError):
        gdn.gdn_linear_attention(t, t, t, torch.zeros(2), t)
    with pytest.raises(TypeError):
        gdn.gdn_rotary(t, None, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))


def test_rotary_frequencies():
    f = gdn.rotary_frequencies(64, 500.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    assert torch.allclose(f, 500.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-14)
    assert torch.allclose(gdn.rotary_frequencies(64, 500.0, scaling="linear", factor=8.0, device="cpu"), f / 8, rtol=1e-14)
    b = gdn.rotary_frequencies(64, 500.0, scaling="base", factor=8.0, device="cpu")
    assert b[0] == 1.0 and math.isclose(float(b[-1]), float(f[-1]) / 8, rel_tol=1e-12)
    p = gdn.rotary_frequencies(64, 500.0, scaling="parts", factor=8.0, original_length=512, device="cpu")
    turns = 512 * f / (2 * math.pi)
    fast, slow = turns > 32, turns < 1
    assert fast.any() and slow.any() and torch.equal(p[fast], f[fast]) and torch.allclose(p[slow], f[slow] / 8, rtol=1e-14)
    mid = ~fast & ~slow
    assert (p[mid] < f[mid]).all() and (p[mid] > f[mid] / 8).all()
    for bad in ({"rotary_dim": 7}, {"rotary_dim": 8, "scaling": "other"}, {"rotary_dim": 8, "scaling": "parts"},
                {"rotary_dim": 8, "scaling": "linear", "factor": 0.0}):
        with pytest.raises(ValueError):
            gdn.rotary_frequencies(device="cpu", **bad)
