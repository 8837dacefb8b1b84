"""Gradients where a sequence ends in a token of garbage that nothing learns from: its x is NaN or infinite and its dy
zero. By the formula dA sums dt_t dh_t exp(dt_t A) h_{t-1}, which holds the state before each token, so the state behind the
last token does not enter: dA stays finite and right whatever the sequence's length, and so do the gradients of all
tokens before. Bounds as in scan_cases."""
import numpy as np
import pytest
import torch

import scan_cases as sc
import ssm_recurrent_decode_gb300 as gdn
import test_parity_scan as scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[1], [5], [8], [13], [70, 9, 64], [300, 3]], ids=str)
@pytest.mark.parametrize("dtype,N", [("f32", 16), ("bf16", 16), ("bf16", 4), ("f32", 128), ("bf16", 24)])
@pytest.mark.parametrize("garbage", [np.nan, np.inf])
def test_garbage_in_the_last_token(lengths, dtype, N, garbage):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    D, T = 40, sum(lengths)
    c = sc.make(lengths, D, N, dtype, 70 + T, skip=False, states=False)
    last = np.cumsum(lengths) - 1
    c["dy"][last] = 0.0
    clean = {k: None if v is None else v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
    clean["x"][last] = 0.0                               # what the formula's sums see: the token's own terms have dy = 0
    ref, mag = sc.backward(clean)
    c["x"][last] = garbage
    d = scan._dev(c, dtype)
    t = scan.TYPES[dtype]
    new = lambda *s, dtype=torch.float32: torch.full(s, 5.0, dtype=dtype, device="cuda")
    g = {"dx": new(T, D, dtype=t), "ddt": new(T, D, dtype=t), "dBm": new(T, N, dtype=t), "dCm": new(T, N, dtype=t), "dA": new(D, N)}
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], z=d["z"], cu_seqlens=scan._cu(lengths),
                                      workspace=scan._workspace(lengths, D, N, False, True), **g)
    torch.cuda.synchronize()
    u = 2 * sc.unit(c)
    before = np.setdiff1d(np.arange(T), last)
    for k, terms in (("dx", 0), ("ddt", 0), ("dBm", D), ("dCm", D)):
        sc.check(k, g[k].float().cpu().numpy()[before], ref[k][before], mag[k][before], u, t, terms)
    sc.check("dx", g["dx"].float().cpu().numpy()[last], ref["dx"][last], mag["dx"][last], u, t)
    sc.check("dA", g["dA"].cpu().numpy(), ref["dA"], mag["dA"], u, terms=T)
