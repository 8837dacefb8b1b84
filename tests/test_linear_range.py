"""Linear attention with states near the ends of fp32's range, under decays that forget within a few tokens: nothing may become
infinite or lose its digits that the recurrence itself keeps."""
import numpy as np
import pytest
import torch

import linear_cases as lc
from test_parity_linear import compare, run_backward, run_forward

pytestmark = pytest.mark.gpu


def _decays(kind, T, HV):
    r = np.random.default_rng(3)
    if kind == "mixed":          # from block to block of 16 tokens: none, weak, and all but the token itself
        g = -np.exp(r.uniform(np.log(1e-3), np.log(40.0), size=(T // 8 + 1, HV))).repeat(8, 0)[:T]
        g[::37] = 0.0
    else:
        g = np.full((T, HV), -float(kind))
    return g.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["0.02", "0.5", "1.1", "1.7", "2.5", "mixed"])
@pytest.mark.parametrize("size", [58, -44])
def test_states_of_any_size(size, decay, dtype):
    """k and v 2^58: products and states of 2^116 and more (fp32 ends at 2^128). 2^-44: of 2^-88, under decays that are
    not so strong that a row's share of them would pass 2^-126 itself."""
    lengths, H, HV, K, V = [150, 75], 1, 2, 32, 24
    c = lc.make(lengths, H, HV, K, V, dtype, 5)
    c["g"] = _decays(decay, sum(lengths), HV)
    f = 2.0 ** size
    for n in ("k", "v"):
        c[n] *= f
    c["q"] /= f
    c["initial"] *= f * f
    c["d_final"] /= f
    refs = lc.references(c)
    compare(c, run_forward(c), refs)
    if size > 0:
        compare(c, run_backward(c), refs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["0.01", "0.2", "runs", "tokens", "mixed"])
def test_log_decays_above_zero(kind, dtype):
    """States that grow, in all tokens or in some of them, while no sum of the log decays leaves +-87 (fp32's powers of two): by 3
    and by 60 over the sequence, in runs of eight tokens to and fro, in every other token, at random."""
    lengths, H, HV, K, V = [300, 77], 1, 2, 64, 48
    c = lc.make(lengths, H, HV, K, V, dtype, 9)
    t, T = np.arange(sum(lengths))[:, None] + np.zeros((1, HV)), sum(lengths)
    g = {"runs": np.where(t // 8 % 2 == 0, -8.0, 8.0), "tokens": np.where(t % 2 == 0, -4.0, 4.0),
         "mixed": 2.0 * np.random.default_rng(2).normal(size=(T, HV)) - 0.5}.get(kind)
    c["g"] = (np.full((T, HV), float(kind)) if g is None else g).astype(np.float32).astype(np.float64)
    refs = lc.references(c)
    forward, backward = run_forward(c), run_backward(c)
    compare(c, forward, refs)
    compare(c, backward, refs)
    for n, x in (("final", forward["final"]), ("d_initial", backward["d_initial"])):
        # a power of two of 87 octaves is a product of a few roundings; from one fp32 number its error would be 87 2^-24
        off = np.linalg.norm(x.double().cpu().numpy() - refs[0][n]) / np.linalg.norm(refs[0][n])
        assert off < 2.0 ** -20, (n, off)
