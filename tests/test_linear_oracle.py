"""The linear-attention references on the CPU: gradients against central differences (whose own error is of order
eps^2 + 2^-53 / eps, taken at eps = 1e-5), and the identities that the kernels use."""
import numpy as np
import pytest

import linear_cases as lc


def _loss(c):
    r = lc.forward(c)
    return float((r["o"] * c["do"]).sum() + (0 if c["d_final"] is None else (r["final"] * c["d_final"]).sum()))


@pytest.mark.parametrize("lengths,H,HV,fixed,states", [([3, 0, 4], 1, 2, False, True), ([5], 2, 2, True, False),
                                                       ([1, 2], 1, 1, True, True)])
def test_gradients_agree_with_differences(lengths, H, HV, fixed, states):
    c = lc.make(lengths, H, HV, 3, 2, "f32", 4, fixed=fixed, states=states)
    b, eps = lc.backward(c), 1e-5
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("initial", "d_initial")):
        if c[name] is None:
            continue
        flat, g = c[name].reshape(-1), b[grad].reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + eps
            up = _loss(c)
            flat[i] = keep - eps
            down = _loss(c)
            flat[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) <= 1e-8 * (1 + abs(g[i])) * 10, (name, i)


def test_the_decays_gradient_telescopes():
    """dg_t = sum over the tokens from t on of q.dq - k.dk, plus <d_final, S_last>."""
    c = lc.make([6, 9], 2, 4, 5, 3, "f32", 8)
    b, f = lc.backward(c), lc.forward(c)
    wide = lambda x: np.repeat(x, 2, 1)
    terms = (wide(c["q"]) * b["dq_heads"]).sum(-1) - (wide(c["k"]) * b["dk_heads"]).sum(-1)
    at = 0
    for s, n in enumerate(c["lengths"]):
        end = (c["d_final"][s] * f["final"][s]).sum((1, 2))
        assert np.allclose(terms[at:at + n][::-1].cumsum(0)[::-1] + end, b["dg"][at:at + n], rtol=1e-10, atol=1e-10)
        at += n


def test_turning_back_is_the_transpose():
    r = np.random.default_rng(1)
    x, y, p, f = r.normal(size=(4, 2, 12)), r.normal(size=(4, 2, 12)), np.array([0, 5, 900, 3]), np.array([1.0, 0.1, 0.01])
    for inter in (False, True):
        a = (lc.turn(x, p, f, 1.3, inter) * y).sum()
        b = (x * lc.turn(y, p, f, 1.3, inter, inverse=True)).sum()
        assert abs(a - b) < 1e-12
