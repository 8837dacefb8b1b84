"""Guard bands and the index-checking build for the sequence and search operators: every written buffer (outputs,
states, gradients, workspaces, pools) lies between canary bytes that must survive, the results equal those on plain
buffers bit for bit, and the debug build's index checks stay silent on the ragged cases and change no result."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import scan_cases as sc
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu

GUARD = 4096
CANARY = 0xA5


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Buffers:
    """Makes plain tensors, or guarded ones (every tensor between two bands of canary bytes)."""

    def __init__(self, guarded):
        self.guarded, self.raws = guarded, []

    def __call__(self, t):
        if not self.guarded or t is None:
            return t
        nbytes = t.numel() * t.element_size()
        raw = torch.full((2 * GUARD + nbytes,), CANARY, dtype=torch.uint8, device="cuda")
        self.raws.append((raw, nbytes))
        v = raw[GUARD:GUARD + nbytes].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    def intact(self):
        torch.cuda.synchronize()
        return all(bool((r[:GUARD] == CANARY).all()) and bool((r[GUARD + n:] == CANARY).all()) for r, n in self.raws)


def _three_ways(run):
    """run(put, err) -> tensors: plain, guarded and on the debug build must agree bit for bit."""
    plain = run(Buffers(False), None)
    guarded = Buffers(True)
    got = run(guarded, None)
    assert guarded.intact(), "bytes outside a buffer were written"
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    with gdn.using_debug_build():
        dbg = run(Buffers(False), err)
    torch.cuda.synchronize()
    assert int(err.item()) & gdn.GDN_DEVERR_RANGE == 0, "a debug index check fired"
    for a, b, c in zip(plain, got, dbg):
        raw = lambda t: t.contiguous().view(-1).view(torch.uint8)
        assert torch.equal(raw(a), raw(b)) and torch.equal(raw(a), raw(c))


CASES = [([5, 0, 70, 1], 37, 13, "f32"), ([33, 20], 65, 16, "bf16"), ([100, 3, 150], 24, 64, "bf16"),
         ([64, 1, 0, 127], 200, 16, "f32"), ([90], 70, 128, "bf16"), ([40, 41], 130, 4, "f32")]


def _put(c, dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    d = {k: None if c[k] is None else torch.from_numpy(c[k]).cuda().to(t) for k in ("x", "dt", "Bm", "Cm", "z", "dy")}
    return d | {k: torch.from_numpy(c[k]).cuda() for k in ("A", "Dskip", "h0", "dh_last")}, t


def _workspace(put, lengths, D, N, backward):
    ws = gdn.mamba_scan_workspace(sum(lengths), D, N, sequences=len(lengths), uniform=False, backward=backward)
    return None if ws is None else put(ws.zero_())


@pytest.mark.parametrize("lengths,D,N,dtype", CASES)
def test_scan(lengths, D, N, dtype):
    c = sc.make(lengths, D, N, dtype, 41)
    d, t = _put(c, dtype)
    T = sum(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    idx = torch.arange(len(lengths), dtype=torch.int32, device="cuda").flip(0).contiguous()

    def run(put, err):
        y, last = put(torch.zeros(T, D, dtype=t, device="cuda")), put(torch.zeros(len(lengths) + 1, D, N, device="cuda"))
        gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], cu_seqlens=cu,
                                 state_indices=idx, h0=torch.cat([d["h0"], d["h0"][:1]]), h_last=last,
                                 workspace=_workspace(put, lengths, D, N, False), err_flags=err)
        return [y, last]

    _three_ways(run)


@pytest.mark.parametrize("lengths,D,N,dtype", CASES)
def test_scan_backward(lengths, D, N, dtype):
    c = sc.make(lengths, D, N, dtype, 42)
    d, t = _put(c, dtype)
    T = sum(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")

    def run(put, err):
        new = lambda *s, dtype=t: put(torch.zeros(*s, dtype=dtype, device="cuda"))
        f32 = torch.float32
        g = {"dx": new(T, D), "ddt": new(T, D), "dz": new(T, D), "dBm": new(T, N), "dCm": new(T, N),
             "dA": new(D, N, dtype=f32), "dDskip": new(D, dtype=f32), "dh0": new(len(lengths), D, N, dtype=f32)}
        gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                          cu_seqlens=cu, h0=d["h0"], dh_last=d["dh_last"],
                                          workspace=_workspace(put, lengths, D, N, True), err_flags=err, **g)
        return list(g.values())

    _three_ways(run)


@pytest.mark.parametrize("batch,beams,V,K,dtype", [(1, 1, 1, 1, "f32"), (3, 4, 50021, 8, "bf16"), (2, 5, 999, 64, "f32"),
                                                   (2, 32, 8191, 33, "bf16")])
def test_select(batch, beams, V, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(43)
    logits = torch.randn(batch * beams, V, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    scores = -torch.rand(batch, beams, generator=g, device="cuda")

    def run(put, err):
        out = [put(torch.zeros(batch, K, device="cuda")), put(torch.zeros(batch, K, dtype=torch.int32, device="cuda")),
               put(torch.zeros(batch, K, dtype=torch.int32, device="cuda")), put(torch.zeros(batch, K, dtype=torch.uint8, device="cuda"))]
        ws = put(gdn.beam_select_workspace(batch, beams, V, K).zero_())
        gdn.gdn_beam_select(logits, scores, *out[:3], out_finished=out[3], eos_token=0, workspace=ws, err_flags=err)
        return out

    _three_ways(run)


def test_reorder():
    r = np.random.default_rng(44)
    batch, beams = 5, 6
    slots = r.permutation(batch * beams + 1)[:batch * beams].reshape(batch, beams).astype(np.int32)
    parents = r.integers(-1, beams, size=(batch, beams)).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(44)
    first = [torch.randn(31, n, generator=g, device="cuda") for n in (5, 4096, 7001)] + \
            [torch.randn(31, 33, generator=g, device="cuda").to(torch.bfloat16)]

    def run(put, err):
        pools = [put(p.clone()) for p in first]
        new = put(torch.zeros(batch, beams, dtype=torch.int32, device="cuda"))
        gdn.gdn_beam_reorder(pools, torch.from_numpy(slots).cuda(), torch.from_numpy(parents).cuda(), new, err_flags=err)
        return pools + [new]

    _three_ways(run)
    assert ref.reorder(slots, parents)[0].shape == slots.shape
