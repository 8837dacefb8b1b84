"""The gradient of the initial state where a sequence starts from zero (dh0 without h0)."""
import numpy as np
import pytest
import torch

import scan_cases as sc
import ssm_recurrent_decode_gb300 as gdn
import test_parity_scan as scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[0], [7], [5, 0, 70, 1], [300, 64]], ids=str)
@pytest.mark.parametrize("dtype,N", [("f32", 16), ("bf16", 4), ("bf16", 50)])
@pytest.mark.parametrize("final", [False, True])
def test_gradient_of_a_zero_initial_state(lengths, dtype, N, final):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    D, T, S = 37, sum(lengths), len(lengths)
    c = sc.make(lengths, D, N, dtype, 80 + T)
    c["h0"] = np.zeros_like(c["h0"])
    if not final:
        c["dh_last"] = np.zeros_like(c["dh_last"])
    d = scan._dev(c, dtype)
    rows = torch.arange(S, dtype=torch.int32, device="cuda").flip(0).contiguous()
    pool = torch.full((S + 1, D, N), 9.0, device="cuda")
    dh_last = torch.zeros_like(pool)
    dh_last[rows.long()] = torch.from_numpy(c["dh_last"]).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dA = torch.empty(D, N, device="cuda")
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                      cu_seqlens=scan._cu(lengths), state_indices=rows, dh_last=dh_last if final else None,
                                      dh0=pool, dA=dA, workspace=scan._workspace(lengths, D, N, False, True), err_flags=err)
    torch.cuda.synchronize()
    ref, mag = sc.backward(c)
    u = 2 * sc.unit(c)
    sc.check("dh0", pool[rows.long()].cpu().numpy(), ref["dh0"], mag["dh0"], u)
    sc.check("dA", dA.cpu().numpy(), ref["dA"], mag["dA"], u, terms=T)
    assert torch.all(pool[S] == 9.0) and int(err.item()) == 0
