"""The selective scan's references on the CPU: the scan is the decode step token by token, and its
gradients agree with central differences of it (fp64; the differences' own error is of order
eps^2 + 2^-53 / eps, taken at eps = 1e-5)."""
import numpy as np
import pytest

import oracle
import scan_cases as sc


def _loss(c, dy, dh_last):
    y, h = oracle.mamba_scan(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], lengths=c["lengths"], Dskip=c["Dskip"],
                             z=c["z"], h0=c["h0"])
    return float((y * dy).sum() + (0 if dh_last is None else (h * dh_last).sum()))


@pytest.mark.parametrize("lengths,gate,skip,states", [([3, 0, 4], True, True, True), ([5], False, False, False),
                                                      ([1, 1], True, False, True)])
def test_gradients_agree_with_differences(lengths, gate, skip, states):
    c = sc.make(lengths, 3, 2, "f32", 5, gate=gate, skip=skip, states=states)
    for k, v in c.items():
        if isinstance(v, np.ndarray):
            c[k] = v.astype(np.float64)
    grads = oracle.mamba_scan_backward(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], lengths=c["lengths"],
                                       Dskip=c["Dskip"], z=c["z"], h0=c["h0"], dh_last=c["dh_last"])
    eps = 1e-5
    for name in ("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "h0"):
        if c[name] is None:
            continue
        flat, g = c[name].reshape(-1), grads["d" + name].reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + eps
            up = _loss(c, c["dy"], c["dh_last"])
            flat[i] = keep - eps
            down = _loss(c, c["dy"], c["dh_last"])
            flat[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) <= 1e-7 * max(1.0, abs(g[i])), (name, i)


def test_scan_is_the_decode_step_token_by_token():
    c = sc.make([4], 5, 3, "f32", 6)
    y, h = oracle.mamba_scan(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], lengths=[4], Dskip=c["Dskip"], z=c["z"], h0=c["h0"])
    s = c["h0"].astype(np.float64)
    for t in range(4):
        r = slice(t, t + 1)
        want = oracle.mamba_decode(c["x"][r], c["dt"][r], c["A"], c["Bm"][r], c["Cm"][r], s, Dskip=c["Dskip"], z=c["z"][r])
        np.testing.assert_array_equal(y[r], want)
    np.testing.assert_array_equal(h, s)


def test_empty_sequences_pass_their_state_and_its_gradient_on():
    c = sc.make([0, 2, 0], 3, 2, "f32", 7)
    y, h = oracle.mamba_scan(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], lengths=c["lengths"], h0=c["h0"])
    np.testing.assert_array_equal(h[[0, 2]], c["h0"][[0, 2]])
    g = oracle.mamba_scan_backward(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], lengths=c["lengths"], h0=c["h0"],
                                   dh_last=c["dh_last"])
    np.testing.assert_array_equal(g["dh0"][[0, 2]], c["dh_last"][[0, 2]])
