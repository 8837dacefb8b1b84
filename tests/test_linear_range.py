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
