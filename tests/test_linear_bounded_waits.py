"""Waits of linear attention's pipelined kernel (bf16 sequences) that give up. The limit is cut to so few SM cycles that
copies, products or other warps' work cannot be done in time: the calls return normally, raise GDN_DEVERR_TIMEOUT, and every output,
state and gradient is either the right one, bit for bit, or NaN; nothing outside the outputs is written. With the default limit
the same calls are exact again. No GPU fault is caused: a kernel whose waits run out ends by itself."""
import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn
from test_linear_machine import Guarded, _random


def test_the_limit_round_trips():
    L = gdn.lib()
    before = L.gdn_linear_set_wait_limit(0)
    assert L.gdn_linear_set_wait_limit(4096) == 0
    assert L.gdn_linear_set_wait_limit(-5) == 4096           # non-positive restores the default
    assert L.gdn_linear_set_wait_limit(1 << 40) == 0
    assert L.gdn_linear_set_wait_limit(0) == 1 << 30         # no longer than the default
    L.gdn_linear_set_wait_limit(before)


def _off_the_grid(t):
    """t in rows that start two bytes past their alignment: a warp copies such tiles by plain loads, in several microseconds each."""
    T, h, n = t.shape
    rows = torch.zeros(T, 1 + h * n, dtype=t.dtype, device="cuda")
    view = rows[:, 1:].unflatten(1, (h, n))
    view.copy_(t)
    return view


def _calls(x, S, err):
    T, H, K = x["q"].shape
    HV, V = x["v"].shape[1:]
    like = {"o": "v", "final": "initial", "dq": "q", "dk": "k", "dv": "v", "dg": "g", "d_initial_state": "initial"}
    b = {n: Guarded(torch.zeros(x[i].shape, dtype=x[i].dtype, device="cuda")) for n, i in like.items()}
    space = lambda w: gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, backward=w)
    args, kw = (x["q"], x["k"], x["v"], x["g"]), {"sequences": S, "initial_state": x["initial"], "err_flags": err, "prepare": True}
    ws = [space(False), space(True)]
    fwd = gdn.gdn_linear_attention(*args, b["o"].t, final_state=b["final"].t, workspace=ws[0], **kw)
    bwd = gdn.gdn_linear_attention_backward(*args, x["do"], d_final_state=x["d_final"], workspace=ws[1], **kw,
                                            **{n: g.t for n, g in b.items() if n.startswith("d")})
    return fwd, bwd, b, [w for w in ws if w is not None]


@pytest.mark.gpu
@pytest.mark.parametrize("S,L,H,HV,K,V,aligned", [
    (3, 300, 2, 2, 128, 128, True),        # whole sequences: one kernel forwards; dq, dk and dv, which starts in dk's last CTAs
    (1, 3000, 2, 4, 64, 128, True),        # cut into segments (a kernel without outputs first), shared heads
    (2, 400, 1, 2, 128, 50, True),         # rows copied to aligned ones
    (2, 900, 2, 2, 128, 128, False),       # slow copies: the waits for them cannot all end in time
])
@pytest.mark.parametrize("limit", [1, 500, 4000, 12000, 40000])
def test_waits_that_run_out_leave_nan(limit, S, L, H, HV, K, V, aligned):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    x = _random(S, L, H, HV, K, V, "bf16", 11 + L)
    if not aligned:
        x |= {n: _off_the_grid(x[n]) for n in ("q", "k", "v", "do")}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fwd, bwd, b, spaces = _calls(x, S, err)
    fwd(), bwd()
    torch.cuda.synchronize()
    assert int(err) == 0
    want = {n: g.t.clone() for n, g in b.items()}
    lib, before = gdn.lib(), gdn.lib().gdn_linear_set_wait_limit(0)
    for call, names in ((fwd, ("o", "final")), (bwd, ("dq", "dk", "dv", "dg", "d_initial_state"))):
        for n in names:
            b[n].t.fill_(3.0)
        for w in spaces:
            w.fill_(0x11)                                   # stale values that must not reach an output
        err.zero_()
        lib.gdn_linear_set_wait_limit(limit)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            lib.gdn_linear_set_wait_limit(before)
        lost = 0
        for n in names:
            nan = b[n].t.isnan()
            lost += int(nan.sum())
            assert bool((nan | (b[n].t == want[n])).all()), n
        assert (int(err) == gdn.GDN_DEVERR_TIMEOUT) == (lost > 0)
        assert lost > 0 or aligned or limit > 500
        assert all(g.intact() for g in b.values())
    err.zero_()
    fwd(), bwd()
    torch.cuda.synchronize()
    assert int(err) == 0
    for n, g in b.items():
        assert torch.equal(g.t, want[n]), n
