"""GPU parity of mamba_selective_scan and mamba_selective_scan_backward against the fp64 references, within the
bounds that scan_cases derives, and their handling of edges: empty and one-token sequences, chunk borders,
odd sizes and strides, states in a pool (also in place), bad indices, streams and graphs."""
import numpy as np
import pytest
import torch

import scan_cases as sc
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _dev(c, dtype, strided=False):
    """Device tensors of a case; strided: odd row strides and an odd first element (no 16-byte rows)."""
    def put(a, t):
        if a is None:
            return None
        v = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t)
        if strided:
            wide = torch.full((v.shape[0] + 1, v.shape[1] + 3), float("nan"), dtype=t, device="cuda")
            wide[:-1, 1:-2] = v
            return wide[:-1, 1:-2]
        return v
    t = TYPES[dtype]
    d = {k: put(c[k], t) for k in ("x", "dt", "Bm", "Cm", "z", "dy")}
    d |= {k: None if c[k] is None else torch.from_numpy(c[k]).cuda() for k in ("A", "Dskip")}
    return d


def _pool(states, S, D, N, seed):
    """A pool [S + 2, D, N] holding `states` at permuted rows, and the rows."""
    rows = np.random.default_rng(seed).permutation(S + 2)[:S].astype(np.int32)
    pool = torch.full((S + 2, D, N), 7.0, device="cuda")
    if states is not None:
        pool[torch.from_numpy(rows).long().cuda()] = torch.from_numpy(states).cuda()
    return pool, torch.from_numpy(rows).cuda()


def _rest(pool, rows):
    keep = torch.ones(pool.shape[0], dtype=torch.bool)
    keep[rows.cpu().long()] = False
    return pool.cpu()[keep]


def _workspace(lengths, D, N, uniform, backward=False):
    ws = gdn.mamba_scan_workspace(sum(lengths), D, N, sequences=len(lengths), uniform=uniform, backward=backward)
    if ws is not None:
        ws.fill_(0xFF)                       # NaN: nothing may be read before it is written
    return ws


def _forward(lengths, D, N, dtype, *, gate=True, skip=True, states=True, uniform=False, out="f32", strided=False,
             in_place=False, seed=0):
    c = sc.make(lengths, D, N, dtype, seed, gate=gate, skip=skip, states=states)
    d = _dev(c, dtype, strided)
    T, S = sum(lengths), len(lengths)
    y = torch.full((T, D), float("nan"), dtype=TYPES[out], device="cuda")
    pool, rows = _pool(c["h0"], S, D, N, seed)
    last = pool if in_place else torch.full_like(pool, 9.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"],
                             sequences=S if uniform else None, cu_seqlens=None if uniform else _cu(lengths),
                             state_indices=rows, h0=pool if states else None, h_last=last,
                             workspace=_workspace(lengths, D, N, uniform), err_flags=err)
    torch.cuda.synchronize()
    ref, mag = sc.forward(c)
    u = sc.unit(c)
    sc.check("y", y.float().cpu().numpy(), ref["y"], mag["y"], u, TYPES[out])
    sc.check("h_last", last[rows.long()].cpu().numpy(), ref["h_last"], mag["h_last"], u)
    assert torch.all(_rest(last, rows) == (7.0 if in_place else 9.0)), "a row of no sequence was written"
    assert int(err.item()) == 0


# ------------------------------------------------------------------------------------------------
# forward
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("N", [1, 3, 4, 8, 13, 16, 24, 32, 50, 64, 100, 128])
def test_state_sizes(N):
    _forward([5, 0, 70, 1], 37, N, "f32", seed=N)


@pytest.mark.parametrize("D", [1, 7, 64, 65, 200])
def test_channel_counts(D):
    _forward([33, 20], D, 16, "bf16", seed=D, out="bf16")


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 1, 0], [15], [16], [17], [31, 1, 32], [32, 32], [64, 1, 0, 63],
                                     [200], [1] * 40, [100, 3, 150]], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths_and_chunk_borders(lengths, dtype):
    _forward(lengths, 24, 16, dtype, seed=sum(lengths))


@pytest.mark.parametrize("gate,skip,states", [(False, False, False), (True, False, False), (False, True, True)])
def test_optional_inputs(gate, skip, states):
    _forward([40, 9], 64, 16, "bf16", gate=gate, skip=skip, states=states, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows(dtype):
    _forward([50, 30], 61, 15, dtype, strided=True, seed=4, out=dtype)


@pytest.mark.parametrize("S,L", [(1, 300), (3, 20), (2, 160), (100, 5), (2, 0)])
def test_equal_lengths(S, L):
    _forward([L] * S, 72, 16, "f32", uniform=True, seed=L)


@pytest.mark.parametrize("lengths,uniform", [([300], True), ([90, 0, 140], False), ([5, 6], False)])
def test_states_in_place(lengths, uniform):
    _forward(lengths, 64, 16, "f32", uniform=uniform, in_place=True, seed=8)


def test_three_axes_and_no_states():
    c = sc.make([12, 12], 40, 16, "f32", 9, states=False)
    d = {k: None if c[k] is None else torch.from_numpy(c[k]).cuda() for k in ("x", "dt", "Bm", "Cm", "z", "A", "Dskip")}
    xz = torch.randn(2, 12, 80, device="cuda")
    xz[..., :40] = d["x"].view(2, 12, 40)
    y = torch.empty(2, 12, 40, device="cuda")
    gdn.mamba_selective_scan(xz[..., :40], d["dt"].view(2, 12, 40), d["A"], d["Bm"].view(2, 12, 16), d["Cm"].view(2, 12, 16),
                             y, Dskip=d["Dskip"], z=d["z"].view(2, 12, 40))
    ref, mag = sc.forward(c)
    sc.check("y", y.view(24, 40).cpu().numpy(), ref["y"], mag["y"], sc.unit(c))


def test_zero_steps_leave_the_state_as_it_is():
    D, N, T = 64, 16, 100
    x, dt = torch.randn(T, D, device="cuda"), torch.zeros(T, D, device="cuda")
    B = torch.randn(T, N, device="cuda")
    h = torch.randn(1, D, N, device="cuda")
    last, y = torch.empty_like(h), torch.empty(T, D, device="cuda")
    A = -torch.rand(D, N, device="cuda") * 100
    gdn.mamba_selective_scan(x, dt, A, B, B, y, h0=h, h_last=last, workspace=gdn.mamba_scan_workspace(T, D, N))
    assert torch.equal(h, last)


def test_prompt_then_decode_equals_one_scan():
    """The state after a prompt, continued by the decode step, against the scan over both."""
    c = sc.make([50], 128, 16, "f32", 10, states=False)
    d = _dev(c, "f32")
    y_all, h_all = torch.empty(50, 128, device="cuda"), torch.empty(1, 128, 16, device="cuda")
    gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y_all, Dskip=d["Dskip"], z=d["z"], h_last=h_all)
    h = torch.empty(1, 128, 16, device="cuda")
    y = torch.empty(50, 128, device="cuda")
    gdn.mamba_selective_scan(d["x"][:40], d["dt"][:40], d["A"], d["Bm"][:40], d["Cm"][:40], y[:40], Dskip=d["Dskip"],
                             z=d["z"][:40], h_last=h)
    for t in range(40, 50):
        gdn.mamba_selective_scan_decode(d["x"][t:t + 1], d["dt"][t:t + 1], d["A"], d["Bm"][t:t + 1], d["Cm"][t:t + 1], h,
                                        y[t:t + 1], Dskip=d["Dskip"], z=d["z"][t:t + 1])
    ref, mag = sc.forward(c)
    for got in (y, y_all):
        sc.check("y", got.cpu().numpy(), ref["y"], mag["y"], sc.unit(c))
    for got in (h, h_all):
        sc.check("h", got.cpu().numpy(), ref["h_last"], mag["h_last"], sc.unit(c))


def test_a_bad_state_index_zeroes_its_sequence_only():
    lengths = [30, 40, 20]
    c = sc.make(lengths, 32, 16, "f32", 11)
    d = _dev(c, "f32")
    h0 = torch.from_numpy(c["h0"]).cuda()
    last = torch.full_like(h0, 9.0)
    y = torch.full((90, 32), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], cu_seqlens=_cu(lengths),
                             state_indices=torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda"), h0=h0, h_last=last,
                             workspace=_workspace(lengths, 32, 16, False), err_flags=err)
    ref, mag = sc.forward(c)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    assert torch.all(y[30:70] == 0) and torch.all(last[1] == 9.0)
    for rows in (slice(0, 30), slice(70, 90)):
        sc.check("y", y[rows].cpu().numpy(), ref["y"][rows], mag["y"][rows], sc.unit(c))
    sc.check("h", last[[0, 2]].cpu().numpy(), ref["h_last"][[0, 2]], mag["h_last"][[0, 2]], sc.unit(c))


def test_nan_stays_in_its_sequence_and_channel():
    lengths = [20, 50, 30]
    c = sc.make(lengths, 32, 16, "f32", 12)
    clean = _dev(c, "f32")
    x = clean["x"].clone()
    x[25, 7] = float("nan")
    out = []
    for xs in (clean["x"], x):
        y, last = torch.empty(100, 32, device="cuda"), torch.empty(3, 32, 16, device="cuda")
        gdn.mamba_selective_scan(xs, clean["dt"], clean["A"], clean["Bm"], clean["Cm"], y, z=clean["z"], cu_seqlens=_cu(lengths),
                                 h0=torch.from_numpy(c["h0"]).cuda(), h_last=last, workspace=_workspace(lengths, 32, 16, False))
        out.append((y, last))
    touched = torch.zeros(100, 32, dtype=torch.bool, device="cuda")
    touched[25:70, 7] = True
    assert torch.all(torch.isnan(out[1][0][touched]))
    assert torch.equal(out[1][0][~touched], out[0][0][~touched])
    assert torch.isnan(out[1][1][1, 7]).all() and torch.equal(out[1][1][[0, 2]], out[0][1][[0, 2]])


def test_infinite_decay_forgets():
    """dt A of minus infinity: the state is the last product alone, also across chunks."""
    T, D, N = 100, 16, 16
    x, B = torch.randn(T, D, device="cuda"), torch.randn(T, N, device="cuda")
    dt = torch.full((T, D), 2.0, device="cuda")
    A = torch.full((D, N), -float("inf"), device="cuda")
    y, last = torch.empty(T, D, device="cuda"), torch.empty(1, D, N, device="cuda")
    gdn.mamba_selective_scan(x, dt, A, B, B, y, h_last=last, cu_seqlens=_cu([T]), workspace=_workspace([T], D, N, False))
    assert torch.equal(last[0], (2.0 * x[-1])[:, None] * B[-1])


def test_on_another_stream_and_in_a_graph():
    lengths = [70, 0, 90]
    c = sc.make(lengths, 64, 16, "bf16", 13)
    d = _dev(c, "bf16")
    h0 = torch.from_numpy(c["h0"]).cuda()
    ws = _workspace(lengths, 64, 16, False)
    cu = _cu(lengths)
    def call(y, last, stream=None):
        gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], cu_seqlens=cu, h0=h0,
                                 h_last=last, workspace=ws, stream=stream)
    new = lambda: (torch.zeros(160, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(h0))
    plain, other, captured = new(), new(), new()
    call(*plain)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(*other, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*captured)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in (other, captured):
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


# ------------------------------------------------------------------------------------------------
# backward
# ------------------------------------------------------------------------------------------------
def _backward(lengths, D, N, dtype, *, gate=True, skip=True, states=True, uniform=False, strided=False, seed=0):
    c = sc.make(lengths, D, N, dtype, seed, gate=gate, skip=skip, states=states)
    d = _dev(c, dtype, strided)
    T, S, t = sum(lengths), len(lengths), TYPES[dtype]
    h0, rows = _pool(c["h0"], S, D, N, seed)
    dh_last, _ = _pool(c["dh_last"], S, D, N, seed)
    def new(*shape, dtype=torch.float32):
        if strided and len(shape) == 2 and dtype is t and shape[0] == T:
            return torch.full((T + 1, shape[1] + 3), float("nan"), dtype=t, device="cuda")[:-1, 1:-2]
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    grads = {"dx": new(T, D, dtype=t), "ddt": new(T, D, dtype=t), "dBm": new(T, N, dtype=t), "dCm": new(T, N, dtype=t),
             "dA": new(D, N), "dz": new(T, D, dtype=t) if gate else None, "dDskip": new(D) if skip else None,
             "dh0": torch.full_like(h0, 9.0) if states else None}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                      sequences=S if uniform else None, cu_seqlens=None if uniform else _cu(lengths),
                                      state_indices=rows, h0=h0 if states else None, dh_last=dh_last if states else None,
                                      workspace=_workspace(lengths, D, N, uniform, True), err_flags=err, **grads)
    torch.cuda.synchronize()
    ref, mag = sc.backward(c)
    u = sc.unit(c)
    # sums one after another: channels of a thread, its lanes, warps and channel tiles (dB, dC); the tokens (dA, dDskip)
    terms = {"dBm": D, "dCm": D, "dA": T, "dDskip": T}
    for k, v in grads.items():
        if v is None:
            continue
        if k == "dh0":
            assert torch.all(_rest(v, rows) == 9.0)
            v = v[rows.long()]
        sc.check(k, v.float().cpu().numpy(), ref[k], mag[k], 2 * u, v.dtype, terms.get(k, 0))
    assert int(err.item()) == 0


@pytest.mark.parametrize("N", [1, 3, 8, 13, 16, 24, 50, 64, 100, 128])
def test_backward_state_sizes(N):
    _backward([5, 0, 70, 1], 37, N, "f32", seed=N)


@pytest.mark.parametrize("D", [1, 7, 64, 65, 200])
def test_backward_channel_counts(D):
    _backward([33, 40], D, 16, "bf16", seed=D)


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 1, 0], [7], [8], [9], [63, 1, 64], [64, 64], [65], [64, 1, 0, 127],
                                     [200], [1] * 70, [100, 3, 150]], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_lengths_and_chunk_borders(lengths, dtype):
    _backward(lengths, 24, 16, dtype, seed=sum(lengths))


@pytest.mark.parametrize("gate,skip,states", [(False, False, False), (True, False, False), (False, True, True)])
def test_backward_optional_inputs(gate, skip, states):
    _backward([40, 59], 64, 16, "bf16", gate=gate, skip=skip, states=states, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_strided_rows(dtype):
    _backward([50, 30], 61, 15, dtype, strided=True, seed=4)


@pytest.mark.parametrize("S,L", [(1, 300), (3, 20), (2, 64), (100, 5), (2, 0)])
def test_backward_equal_lengths(S, L):
    _backward([L] * S, 72, 16, "f32", uniform=True, seed=L)


def test_backward_agrees_with_differences_of_the_forward_call():
    """dA and dh0 against central differences of the GPU forward pass. The loss is a sum of about 10^3 terms of order
    one, each fp32-rounded (off by up to unit(c) of its magnitude); at a step of 2^-6 the differences carry that over
    2^-5, and their own third-order term stays below 2^-12 of the magnitude for |dt| <= 0.3 over 12 tokens."""
    lengths = [12]
    c = sc.make(lengths, 8, 4, "f32", 21, gate=False)
    d = _dev(c, "f32")
    h0, dhl = torch.from_numpy(c["h0"]).cuda(), torch.from_numpy(c["dh_last"]).cuda()
    def loss(A, h):
        y, last = torch.empty(12, 8, device="cuda"), torch.empty_like(h)
        gdn.mamba_selective_scan(d["x"], d["dt"], A, d["Bm"], d["Cm"], y, Dskip=d["Dskip"], h0=h, h_last=last)
        return float((y.double() * d["dy"].double()).sum() + (last.double() * dhl.double()).sum())
    dA, dh0 = torch.empty(8, 4, device="cuda"), torch.empty_like(h0)
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], h0=h0,
                                      dh_last=dhl, dA=dA, dh0=dh0, workspace=gdn.mamba_scan_workspace(12, 8, 4, backward=True))
    _, mag = sc.forward(c)
    size = float((mag["y"] * np.abs(c["dy"])).sum() + (mag["h_last"] * np.abs(c["dh_last"])).sum())
    eps = 2.0 ** -6
    tol = size * (sc.unit(c) / eps + 2.0 ** -12)
    for got, base, i in ((dA, d["A"], (3, 1)), (dA, d["A"], (7, 3)), (dh0, h0, (0, 2, 0)), (dh0, h0, (0, 5, 3))):
        step = torch.zeros_like(base)
        step[i] = eps
        pair = [(d["A"] + s * step, h0) if base is d["A"] else (d["A"], h0 + s * step) for s in (1, -1)]
        diff = (loss(*pair[0]) - loss(*pair[1])) / (2 * eps)
        assert abs(diff - float(got[i])) <= tol, (i, diff, float(got[i]), tol)


def test_backward_writes_only_what_is_asked_for_and_repeats_bitwise():
    lengths = [90, 40]
    c = sc.make(lengths, 64, 16, "bf16", 22)
    d = _dev(c, "bf16")
    def run(names):
        t = {"dx": (130, 64), "ddt": (130, 64), "dz": (130, 64), "dBm": (130, 16), "dCm": (130, 16)}
        g = {k: torch.zeros(t[k], dtype=torch.bfloat16, device="cuda") for k in names if k in t}
        if "dA" in names:
            g["dA"] = torch.zeros(64, 16, device="cuda")
        gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                          cu_seqlens=_cu(lengths), workspace=_workspace(lengths, 64, 16, False, True), **g)
        return g
    full = run(["dx", "ddt", "dz", "dBm", "dCm", "dA"])
    again = run(["dx", "ddt", "dz", "dBm", "dCm", "dA"])
    for k in full:
        assert torch.equal(full[k], again[k]), k
    for k in full:
        assert torch.equal(run([k])[k], full[k]), k


def test_backward_a_bad_state_index_zeroes_its_sequence_only():
    lengths = [30, 70, 20]
    c = sc.make(lengths, 32, 16, "f32", 23)
    d = _dev(c, "f32")
    h0, dhl = torch.from_numpy(c["h0"]).cuda(), torch.from_numpy(c["dh_last"]).cuda()
    g = {"dx": torch.full((120, 32), 5.0, device="cuda"), "dBm": torch.full((120, 16), 5.0, device="cuda"),
         "dA": torch.empty(32, 16, device="cuda"), "dh0": torch.full_like(h0, 9.0)}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                      cu_seqlens=_cu(lengths), state_indices=torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda"),
                                      h0=h0, dh_last=dhl, workspace=_workspace(lengths, 32, 16, False, True), err_flags=err, **g)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    assert torch.all(g["dx"][30:100] == 0) and torch.all(g["dBm"][30:100] == 0) and torch.all(g["dh0"][1] == 9.0)
    parts = [sc.backward({**c, **{k: c[k][r] for k in ("x", "dt", "Bm", "Cm", "z", "dy")}, "lengths": [r.stop - r.start],
                          "h0": c["h0"][i:i + 1], "dh_last": c["dh_last"][i:i + 1]}) for i, r in ((0, slice(0, 30)), (2, slice(100, 120)))]
    u = 2 * sc.unit(c)
    sc.check("dx", g["dx"][:30].cpu().numpy(), parts[0][0]["dx"], parts[0][1]["dx"], u)
    sc.check("dx", g["dx"][100:].cpu().numpy(), parts[1][0]["dx"], parts[1][1]["dx"], u)
    sc.check("dA", g["dA"].cpu().numpy(), parts[0][0]["dA"] + parts[1][0]["dA"], parts[0][1]["dA"] + parts[1][1]["dA"], u, terms=120)


def test_long_chunks():
    """Sizes whose chunks hold many tiles: several hundred rows forward, 64 backward, sequences across them."""
    _forward([2500, 0, 3400, 100], 2000, 16, "bf16", seed=31)
    _backward([500, 1, 700, 0, 99], 2000, 16, "bf16", seed=32)


@pytest.mark.parametrize("N", [3, 16, 24, 50, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_sizes_across_chunks(N, dtype):
    """Calls too long for one cluster of chunks: a summary, a carry and an output launch."""
    _forward([5, 0, 270, 1, 64], 37, N, dtype, seed=N, out=dtype)


@pytest.mark.parametrize("T", [33, 100, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("in_place", [False, True])
def test_short_calls(T, in_place):
    """Calls of a few chunks: one sequence, and one that ends and one that begins inside."""
    _forward([T], 72, 16, "f32", seed=T, in_place=in_place)
    _forward([T // 3, T - T // 3 - 5, 5], 72, 16, "f32", seed=T, in_place=in_place)


@pytest.mark.parametrize("fill", [0x00, 0x01, 0x7F])
def test_what_the_workspace_held_does_not_matter(fill):
    """Several chunks with states in a pool: outputs bit-equal whatever the workspace's bytes were."""
    lengths, D, N = [5, 0, 400, 1, 64], 72, 16
    c = sc.make(lengths, D, N, "bf16", 50)
    d = _dev(c, "bf16")
    h0, rows = _pool(c["h0"], 5, D, N, 50)
    out = []
    for byte in (fill, 0xFF):
        y, last = torch.zeros(470, D, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(h0)
        ws = _workspace(lengths, D, N, False)
        assert ws is not None
        gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], cu_seqlens=_cu(lengths),
                                 state_indices=rows, h0=h0, h_last=last, workspace=ws.fill_(byte))
        dx, dA, dh0 = torch.zeros_like(d["x"]), torch.zeros(D, N, device="cuda"), torch.zeros_like(h0)
        gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                          cu_seqlens=_cu(lengths), state_indices=rows, h0=h0, dh_last=h0, dx=dx, dA=dA, dh0=dh0,
                                          workspace=_workspace(lengths, D, N, False, True).fill_(byte))
        torch.cuda.synchronize()
        out.append((y, last, dx, dA, dh0))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,S", [(60, 2), (300, 3), (30, 1)])
def test_rows_of_no_sequence_are_zero_and_flagged(T, S):
    """cu_seqlens that begin behind row 0 and end before row T - 1: the other rows' outputs and gradients are zeros."""
    D, N, first = 40, 16, 7
    lengths = [(T - 20) // S] * S
    end = first + sum(lengths)
    c = sc.make([T], D, N, "f32", 60, states=False)
    d = _dev(c, "f32")
    cu = torch.tensor(first + np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    y = torch.full((T, D), 5.0, device="cuda")
    ws = gdn.mamba_scan_workspace(T, D, N, sequences=S, uniform=False)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.mamba_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], y, Dskip=d["Dskip"], z=d["z"], cu_seqlens=cu,
                             workspace=ws, err_flags=err)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    g = {"dx": torch.full((T, D), 5.0, device="cuda"), "dCm": torch.full((T, N), 5.0, device="cuda"), "dA": torch.empty(D, N, device="cuda")}
    err.zero_()
    gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"], cu_seqlens=cu,
                                      workspace=gdn.mamba_scan_workspace(T, D, N, sequences=S, uniform=False, backward=True),
                                      err_flags=err, **g)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    inner = {**c, **{k: c[k][first:end] for k in ("x", "dt", "Bm", "Cm", "z", "dy")}, "lengths": lengths}
    (ref, mag), (gref, gmag), u = sc.forward(inner), sc.backward(inner), sc.unit(inner)
    sc.check("y", y[first:end].cpu().numpy(), ref["y"], mag["y"], u)
    sc.check("dx", g["dx"][first:end].cpu().numpy(), gref["dx"], gmag["dx"], 2 * u)
    sc.check("dCm", g["dCm"][first:end].cpu().numpy(), gref["dCm"], gmag["dCm"], 2 * u, terms=D)
    sc.check("dA", g["dA"].cpu().numpy(), gref["dA"], gmag["dA"], 2 * u, terms=T)
    for t in (y, g["dx"], g["dCm"]):
        assert torch.all(t[:first] == 0) and torch.all(t[end:] == 0)
