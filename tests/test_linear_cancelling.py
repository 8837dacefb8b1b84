"""Linear attention in bf16 where a sum's terms cancel: states or values with a common mean, and vectors orthogonal to it. Such
outputs are small beside their terms, so that a state or a score rounded to one bf16 number (2^-8 of a term) on its way
into a product would show, which the header forbids. The bound is the one that linear_cases derives for operands of two bf16
numbers, whatever the outputs' type: ((L + K + V + 32) 2^-23 + 2^-16) of the terms' magnitudes, and half a step of the output."""
import numpy as np
import pytest
import torch

import linear_cases as lc
from test_parity_linear import run_backward, run_forward

pytestmark = pytest.mark.gpu


def _orthogonal(r, T, heads, n):
    """Vectors whose channels sum to zero exactly: neighbours of opposite sign."""
    x = lc.values(np.abs(r.normal(size=(T, heads, n // 2))), "bf16")
    return np.stack([x, -x], -1).reshape(T, heads, n)


def _check(c, got, names, out):
    ref, mag = lc.references(c)
    K, V, L = c["q"].shape[2], c["v"].shape[2], max(c["lengths"])
    for n in names:
        g, half = got[n].double().cpu().numpy(), torch.finfo(got[n].dtype).eps / 2
        tol = ((L + K + V + 32) * 2.0 ** -23 + 2.0 ** -16) * mag[n] * (1 + half) + half * np.abs(ref[n])
        off = np.abs(g - ref[n])
        assert np.all(off <= tol), (n, float(np.max(off / tol)), out)


@pytest.mark.parametrize("H,HV", [(2, 2), (1, 3)])
@pytest.mark.parametrize("only", [None, ("dq", "dk", "dv", "d_initial_state")])
def test_states_with_a_common_mean(only, H, HV):
    """The states that a sequence starts with and whose gradients it ends with are 1 with a spread of 0.02; what
    the tokens add is small beside them."""
    K = V = 16
    c = lc.make([40, 3, 20], H, HV, K, V, "bf16", 5, decay=(1e-3, 1e-2))
    r = np.random.default_rng(6)
    for n in ("q", "k", "v", "do"):
        c[n] = _orthogonal(r, *c[n].shape) / 64
    for n in ("initial", "d_final"):
        c[n] = (1.0 + 0.02 * c[n]).astype(np.float32).astype(np.float64)
    if only is None:
        _check(c, run_forward(c), ("o",), "bf16")
        _check(c, run_forward(c, out="f32"), ("o",), "f32")
    _check(c, run_backward(c, only=only), ("dq", "dk", "dv"), only)


@pytest.mark.parametrize("x,y,z,outs", [("q", "k", "v", ("o",)), ("do", "v", "k", ("dq",)), ("k", "q", "do", ("dv",)), ("v", "do", "q", ("dk",))])
def test_scores_that_cancel(x, y, z, outs):
    """y changes its sign from token to token and z hardly differs: the scores cancel in pairs."""
    K = V = 16
    c = lc.make([20, 18], 1, 1, K, V, "bf16", 7, fixed=True, states=False)
    r = np.random.default_rng(8)
    c["g"] = np.array([np.float32(-0.003)], dtype=np.float64)
    T = c["q"].shape[0]
    for n in ("q", "k", "v", "do"):
        c[n] = lc.values(np.abs(r.normal(size=c[n].shape)), "bf16")
    c[y][1::2] = -c[y][0::2]
    c[z] = lc.values(1.0 + 0.02 * r.normal(size=c[z].shape), "bf16")
    got = run_forward(c) if outs == ("o",) else run_backward(c, only=outs)
    _check(c, got, outs, "bf16")
