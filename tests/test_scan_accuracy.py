"""The selective scan's accuracy over long memories, in relative L2 norm against 64 bits. The bounds of scan_cases grow with
the sequence and would pass a decay that is off by 1e-8 of its value in every token; these do not.

The limits are twice the largest figure of the nine cases beside the decays' constant in scan_common.cuh: 7.0e-7 for
final states and gradients of initial ones, 7.9e-7 for gradients of A, 5.8e-7 for outputs in fp32. Without that
constant the states of the first test are off by 1.7e-6 (with it 6.2e-7). Inputs as a model has them: step sizes of 0.001 to 0.1 about
each channel's own, rates about 1 to N."""
import numpy as np
import pytest
import torch

import oracle
import ssm_recurrent_decode_gb300 as gdn
import test_parity_scan as scan

pytestmark = pytest.mark.gpu

STATES, RATES, OUTPUTS = 2 * 7.0e-7, 2 * 7.9e-7, 2 * 5.8e-7


def inputs(lengths, D, N, seed):
    r = np.random.default_rng(seed)
    T, S = sum(lengths), len(lengths)
    f = lambda *s: r.normal(size=s).astype(np.float32)
    x = f(T, D)
    base = np.exp(r.uniform(np.log(1e-3), np.log(0.1), size=D))
    return {"x": x / (1 + np.exp(-x)), "dt": (base * np.exp(0.5 * r.normal(size=(T, D)))).astype(np.float32), "Bm": f(T, N), "Cm": f(T, N),
            "z": f(T, D), "dy": f(T, D), "Dskip": 1 + 0.1 * f(D), "h0": f(S, D, N), "dh_last": 0.1 * f(S, D, N),
            "A": (-np.arange(1, N + 1) * np.exp(0.1 * r.normal(size=(D, N)))).astype(np.float32), "lengths": list(lengths)}


def off(got, ref):
    return float(np.linalg.norm(got.double().cpu().numpy() - ref) / np.linalg.norm(ref))


def test_states_and_outputs():
    """Sequences of 1024 tokens, each in one pass: a state's decays are multiplied up over all of them."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S, L, D, N = 32, 1024, 64, 128
    c = inputs([L] * S, D, N, 90)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if k != "lengths"}
    y, h = torch.empty(S * L, D, device="cuda"), torch.empty(S, D, N, device="cuda")
    assert gdn.mamba_scan_workspace(S * L, D, N, sequences=S) is None       # nothing is carried between chunks
    gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], h0=d["h0"], h_last=h, sequences=S)
    ry, rh = np.empty((S * L, D)), c["h0"].astype(np.float64)
    for p in range(L):
        t = np.arange(S) * L + p
        ry[t] = oracle.mamba_decode(c["x"][t], c["dt"][t], c["A"], c["Bm"][t], c["Cm"][t], rh, Dskip=c["Dskip"], z=c["z"][t])
    assert off(h, rh) < STATES and off(y, ry) < OUTPUTS


@pytest.mark.parametrize("lengths,D,N", [([2000], 64, 16), ([1000, 1000], 64, 64)])
def test_gradients(lengths, D, N):
    c = inputs(lengths, D, N, 91)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if k != "lengths"}
    dA, dh0 = torch.empty(D, N, device="cuda"), torch.empty(len(lengths), D, N, device="cuda")
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"], h0=d["h0"],
                                      dh_last=d["dh_last"], cu_seqlens=scan._cu(lengths), dA=dA, dh0=dh0,
                                      workspace=scan._workspace(lengths, D, N, False, True))
    ref = oracle.mamba_scan_backward(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], lengths=lengths, Dskip=c["Dskip"], z=c["z"],
                                     h0=c["h0"], dh_last=c["dh_last"])
    assert off(dA, ref["dA"]) < RATES and off(dh0, ref["dh0"]) < STATES
