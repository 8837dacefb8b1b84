"""CPU checks of the selective scan's host side: refusals before any CUDA call, and workspace sizes."""
import ctypes

import pytest

import ssm_recurrent_decode_gb300 as gdn

BASE = 1 << 40


def _valid():
    """Arguments with fake, aligned addresses that are never dereferenced."""
    m = gdn.MambaScanArgs()
    m.T, m.S, m.D, m.N, m.in_dtype, m.out_dtype = 300, 1, 64, 16, gdn.GDN_BF16, gdn.GDN_BF16
    for i, f in enumerate(("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "y", "h0", "h_last", "workspace")):
        setattr(m, f, BASE + (i << 32))
    m.x_stride = m.dt_stride = m.z_stride = m.y_stride = 64
    m.B_stride = m.C_stride = 16
    m.num_states = 1
    m.workspace_bytes = 1 << 30
    return m


REFUSED = [
    ("no x", lambda m: setattr(m, "x", None), -1),
    ("no A", lambda m: setattr(m, "A", None), -1),
    ("no workspace", lambda m: setattr(m, "workspace", None), -1),
    ("negative T", lambda m: setattr(m, "T", -1), -2),
    ("no sequence", lambda m: setattr(m, "S", 0), -2),
    ("no channel", lambda m: setattr(m, "D", 0), -2),
    ("N of zero", lambda m: setattr(m, "N", 0), -2),
    ("N above 128", lambda m: setattr(m, "N", 129), -2),
    ("unequal sequences without cu_seqlens", lambda m: setattr(m, "S", 7), -2),
    ("row stride below the row", lambda m: setattr(m, "dt_stride", 63), -2),
    ("B stride below the row", lambda m: setattr(m, "B_stride", 15), -2),
    ("workspace too small", lambda m: setattr(m, "workspace_bytes", 100), -2),
    ("no state rows", lambda m: setattr(m, "num_states", 0), -2),
    ("fewer state rows than sequences", lambda m: (setattr(m, "S", 2),), -2),
    ("input type", lambda m: setattr(m, "in_dtype", 2), -3),
    ("output type", lambda m: setattr(m, "out_dtype", -1), -3),
    ("x not on an element", lambda m: setattr(m, "x", BASE + 1), -4),
    ("A not on an element", lambda m: setattr(m, "A", BASE + 2), -4),
    ("workspace not on 16 bytes", lambda m: setattr(m, "workspace", BASE + 8), -4),
]


@pytest.mark.parametrize("name,mutate,code", REFUSED, ids=[r[0] for r in REFUSED])
def test_scan_refuses_on_the_host(name, mutate, code):
    m = _valid()
    mutate(m)
    assert gdn.lib().mamba_selective_scan(ctypes.byref(m), None) == code


def _valid_grad():
    a = gdn.MambaScanGradArgs()
    a.s = _valid()
    for i, f in enumerate(("dy", "dh_last", "dx", "ddt", "dz", "dBm", "dCm", "dA", "dDskip", "dh0")):
        setattr(a, f, BASE + ((20 + i) << 32))
    a.dy_stride = a.dx_stride = a.ddt_stride = a.dz_stride = 64
    a.dB_stride = a.dC_stride = 16
    return a


REFUSED_GRAD = [
    ("no dy", lambda a: setattr(a, "dy", None), -1),
    ("no C", lambda a: setattr(a.s, "Cm", None), -1),
    ("dy stride below the row", lambda a: setattr(a, "dy_stride", 1), -2),
    ("dB stride below the row", lambda a: setattr(a, "dB_stride", 8), -2),
    ("workspace too small", lambda a: setattr(a.s, "workspace_bytes", 1000), -2),
    ("input type", lambda a: setattr(a.s, "in_dtype", 5), -3),
    ("dx not on an element", lambda a: setattr(a, "dx", BASE + 1), -4),
    ("dA not on an element", lambda a: setattr(a, "dA", BASE + 2), -4),
    ("dz without z", lambda a: setattr(a.s, "z", None), -6),
    ("dDskip without Dskip", lambda a: setattr(a.s, "Dskip", None), -6),
]


@pytest.mark.parametrize("name,mutate,code", REFUSED_GRAD, ids=[r[0] for r in REFUSED_GRAD])
def test_backward_refuses_on_the_host(name, mutate, code):
    a = _valid_grad()
    mutate(a)
    assert gdn.lib().mamba_selective_scan_backward(ctypes.byref(a), None) == code


def test_null_arguments_and_nothing_to_do():
    L = gdn.lib()
    assert L.mamba_selective_scan(None, None) == -1
    assert L.mamba_selective_scan_backward(None, None) == -1
    m = _valid()
    m.T, m.h_last, m.x = 0, None, None
    assert L.mamba_selective_scan(ctypes.byref(m), None) == 0


def test_workspace_sizes():
    f = gdn.lib().mamba_scan_workspace_bytes
    assert f(100, 1, 64, 16, 1, 0) == 0                    # one short sequence: one pass
    assert f(16384, 64, 1536, 16, 1, 0) == 0               # many sequences of one length: one pass
    assert f(32768, 1, 1536, 16, 1, 0) > 0
    assert f(300, 5, 64, 16, 0, 1) > f(300, 5, 64, 16, 0, 0) > 0
    for bad in ((-1, 1, 64, 16), (10, 0, 64, 16), (10, 3, 64, 16), (10, 1, 0, 16), (10, 1, 64, 129)):
        assert f(*bad, 1, 1) == 0


def test_struct_sizes_and_binding_checks():
    torch = pytest.importorskip("torch")
    L = gdn.lib()
    assert L.gdn_abi_struct_size(6) == ctypes.sizeof(gdn.MambaScanArgs)
    assert L.gdn_abi_struct_size(7) == ctypes.sizeof(gdn.MambaScanGradArgs)
    z = torch.zeros
    with pytest.raises(TypeError, match="CUDA"):
        gdn.mamba_selective_scan(z(4, 8), z(4, 8), z(8, 2), z(4, 2), z(4, 2), z(4, 8))
    with pytest.raises(ValueError, match="rows"):
        gdn._token_rows(z(4, 9), "x", 4, 8)
    with pytest.raises(ValueError, match="inner stride"):
        gdn._token_rows(z(8, 4).t(), "x", 4, 8)
    with pytest.raises(ValueError, match="follow one another"):
        gdn._token_rows(z(2, 6, 8)[:, :4], "x", 8, 8)
