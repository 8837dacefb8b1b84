"""GPU parity of linear attention (prompts, gradients, single tokens) against the 64-bit references, within the bounds
that linear_cases derives, and its edges: empty and one-token sequences, borders of chunks and segments, odd sizes
and strides, states in a pool (also in place), bad indices, rows outside the sequences, NaN, streams and graphs."""
import numpy as np
import pytest
import torch

import linear_cases as lc
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _uniform(c):
    return len(set(c["lengths"])) == 1


def _workspace(c, uniform, backward):
    T, HV, V = c["v"].shape
    H, K = c["q"].shape[1:]
    ws = gdn.linear_attention_workspace(T, H, HV, K, V, sequences=len(c["lengths"]), uniform=uniform, backward=backward,
                                        dtype=lc.TYPES[c["dtype"]])
    if ws is not None:
        ws.fill_(0xFF)                       # NaN: nothing may be read before it is written
    return ws


def _seqs(c, uniform):
    return {"sequences": len(c["lengths"])} if uniform else {"cu_seqlens": lc.cu(c["lengths"])}


def _inputs(c, layout="rows"):
    return [lc.put(c[n], c["dtype"], layout) for n in ("q", "k", "v")] + [lc.f32(c["g"])]


def run_forward(c, *, uniform=None, layout="rows", out="same", in_place=False, err=None, **kw):
    uniform = _uniform(c) if uniform is None else uniform
    S, (T, HV, V), K = len(c["lengths"]), c["v"].shape, c["q"].shape[2]
    q, k, v, g = _inputs(c, layout)
    o = lc.put(np.zeros((T, HV, V)), c["dtype"] if out == "same" else out, layout)
    o.fill_(float("nan"))
    start, rows = lc.pool(c["initial"], S, (HV, V, K), 3)
    final = start if in_place else lc.pool(None, S, (HV, V, K), 3)[0]
    before = lc.rest(final, rows)
    gdn.gdn_linear_attention(q, k, v, g, o, initial_state=None if c["initial"] is None else start, final_state=final,
                             state_indices=rows, workspace=_workspace(c, uniform, False), err_flags=err, **_seqs(c, uniform), **kw)
    torch.cuda.synchronize()
    assert torch.equal(lc.rest(final, rows), before)
    return {"o": o, "final": final[rows.long()]}


def run_backward(c, *, uniform=None, layout="rows", only=None, err=None):
    uniform = _uniform(c) if uniform is None else uniform
    S, (T, HV, V), (H, K) = len(c["lengths"]), c["v"].shape, c["q"].shape[1:]
    q, k, v, g = _inputs(c, layout)
    do = lc.put(c["do"], c["dtype"], layout)
    start, rows = lc.pool(c["initial"], S, (HV, V, K), 3)
    end, _ = lc.pool(c["d_final"], S, (HV, V, K), 3)
    out = {"dq": lc.put(np.zeros((T, H, K)), c["dtype"], layout), "dk": lc.put(np.zeros((T, H, K)), c["dtype"], layout),
           "dv": lc.put(np.zeros((T, HV, V)), c["dtype"], layout), "dg": torch.empty_like(g),
           "d_initial_state": lc.pool(None, S, (HV, V, K), 3)[0]}
    for n in ("dq", "dk", "dv", "dg"):
        out[n].fill_(float("nan"))
    if only is not None:
        out = {n: t for n, t in out.items() if n in only}
    gdn.gdn_linear_attention_backward(q, k, v, g, do, initial_state=None if c["initial"] is None else start,
                                      d_final_state=None if c["d_final"] is None else end, state_indices=rows,
                                      workspace=_workspace(c, uniform, True), err_flags=err, **_seqs(c, uniform), **out)
    torch.cuda.synchronize()
    if "d_initial_state" in out:
        assert bool((lc.rest(out["d_initial_state"], rows) == 7.0).all())
        out["d_initial"] = out.pop("d_initial_state")[rows.long()]
    return out


def compare(c, got, refs=None):
    ref, mag = refs or lc.references(c)
    for n, t in got.items():
        token = n in ("o", "dq", "dk", "dv")
        lc.check(c, n, t, ref[n], mag[n], {torch.float32: "f32", torch.bfloat16: "bf16"}[t.dtype] if token else "f32")


CASES = [
    # lengths, H, HV, K, V, fixed, states
    ([1], 1, 1, 16, 1, False, True),
    ([0, 1, 2, 15, 16, 17], 1, 2, 32, 8, False, True),
    ([64, 63, 65, 1, 0], 2, 2, 64, 64, False, True),
    ([127, 128, 129], 2, 4, 128, 128, False, True),
    ([128, 128], 1, 3, 64, 128, True, False),
    ([300], 2, 2, 128, 50, False, False),
    ([37, 200, 0, 5, 90], 1, 4, 16, 128, True, True),
    ([150], 3, 3, 32, 33, True, True),
    ([700], 1, 1, 64, 24, False, True),
    ([257, 511], 1, 1, 128, 72, True, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,HV,K,V,fixed,states", CASES)
def test_forward(lengths, H, HV, K, V, fixed, states, dtype):
    c = lc.make(lengths, H, HV, K, V, dtype, 11 + sum(lengths), fixed=fixed, states=states)
    compare(c, run_forward(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,HV,K,V,fixed,states", CASES)
def test_backward(lengths, H, HV, K, V, fixed, states, dtype):
    c = lc.make(lengths, H, HV, K, V, dtype, 13 + sum(lengths), fixed=fixed, states=states)
    compare(c, run_backward(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["dense", "odd", "heads"])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 40), (32, 31)])
def test_layouts(K, V, layout, dtype):
    c = lc.make([90, 1, 180], 2, 4, K, V, dtype, 17)
    refs = lc.references(c)
    compare(c, run_forward(c, layout=layout), refs)
    compare(c, run_backward(c, layout=layout), refs)


def test_fp32_outputs_of_bf16_inputs():
    c = lc.make([140, 75], 2, 2, 64, 64, "bf16", 19)
    compare(c, run_forward(c, out="f32"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_states(dtype):
    c = lc.make([400, 3, 0, 130], 1, 2, 64, 48, dtype, 23)
    compare(c, run_forward(c, in_place=True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_by_table_and_by_count_agree(dtype):
    c = lc.make([160, 160, 160], 1, 2, 32, 64, dtype, 29)
    refs = lc.references(c)
    compare(c, run_forward(c, uniform=False), refs)
    compare(c, run_backward(c, uniform=False), refs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("only", [("dq",), ("dk",), ("dv",), ("dg",), ("d_initial_state",), ("dq", "dv")])
def test_single_gradients(only, dtype):
    c = lc.make([100, 31], 1, 2, 32, 40, dtype, 31)
    compare(c, run_backward(c, only=only))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_without_a_given_end(dtype):
    c = lc.make([260, 4], 1, 2, 64, 64, dtype, 37)
    c["d_final"] = None
    compare(c, run_backward(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [(1e-6, 1e-5), (1.0, 50.0), (80.0, 400.0)])
def test_decays(decay, dtype):
    """Long memories, memories of a few tokens, and none."""
    c = lc.make([300, 129], 1, 2, 64, 64, dtype, 41, decay=decay)
    c["g"][10:20] = 0.0
    c["g"] = np.maximum(c["g"], -200.0)
    refs = lc.references(c)
    compare(c, run_forward(c), refs)
    compare(c, run_backward(c), refs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_forgotten_past(dtype):
    """g = -inf cuts a sequence in two: what follows is what a sequence of its own gives."""
    c = lc.make([200], 1, 2, 64, 64, dtype, 43, states=False)
    at = 77
    d = {k: x for k, x in c.items()} | {"lengths": [at, 200 - at]}
    want, mag = lc.forward(d), lc._magnitudes(c)
    grads = lc.backward(d)
    c["g"][at] = -np.inf
    got = run_forward(c)
    lc.check(c, "o", got["o"], want["o"], mag["o"], dtype)
    got = run_backward(c)
    for n in ("dq", "dk", "dv"):
        lc.check(c, n, got[n], grads[n], mag[n], dtype)
    assert bool((got["dg"][at].abs() <= torch.from_numpy((200 + 160) * 2.0 ** -15 * mag["dg"][at]).cuda()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "g"])
def test_nan_stays_behind_its_token(name, dtype):
    """A NaN in one token changes no earlier output, no other sequence, head or (for v) channel."""
    c = lc.make([150, 140], 2, 2, 64, 64, dtype, 47)
    clean = run_forward(c)
    t = 70
    c[name][(t, 0, 5) if name != "g" else (t, 0)] = np.nan
    got = run_forward(c)
    o, want = got["o"].float(), clean["o"].float()
    assert torch.equal(o[:t], want[:t]) and torch.equal(o[150:], want[150:]) and torch.equal(o[:, 1], want[:, 1])
    assert torch.equal(got["final"][1], clean["final"][1]) and torch.equal(got["final"][0, 1], clean["final"][0, 1])
    bad = o[t:150, 0].isnan()
    if name == "q":
        assert bool(bad[0].all()) and torch.equal(o[t + 1:], want[t + 1:]) and torch.equal(got["final"], clean["final"])
    elif name == "v":
        assert bool(bad[:, 5].all()) and int(bad.sum()) == 150 - t
        assert bool(got["final"][0, 0, 5].isnan().all()) and int(got["final"].isnan().sum()) == 64
    else:
        assert bool(bad.all())
        assert bool((got["final"][0, 0].isnan().all() if name == "g" else got["final"][0, 0, :, 5].isnan().all()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_nan_gradients_stay_on_their_side(name, dtype):
    """dq sees earlier tokens only, dk and dv later ones; nothing crosses into another sequence or head."""
    c = lc.make([150, 140], 2, 2, 64, 64, dtype, 53)
    clean = run_backward(c)
    t = 70
    c[name][t, 0, 5] = np.nan
    got = run_backward(c)
    for n in ("dq", "dk", "dv", "dg"):
        assert torch.equal(got[n][150:], clean[n][150:]) and torch.equal(got[n][:, 1], clean[n][:, 1]), n
    if name in ("k", "v"):
        assert torch.equal(got["dq"][:t], clean["dq"][:t])                     # an earlier dq does not read them
        keep = slice(t + 1, 150)
        assert torch.equal(got["dk"][keep], clean["dk"][keep]) and torch.equal(got["dv"][keep], clean["dv"][keep])
    else:
        keep = slice(t + 1, 150)
        assert torch.equal(got["dk"][keep], clean["dk"][keep]) and torch.equal(got["dv"][keep], clean["dv"][keep])
        rest = torch.cat([got["dq"][:t], got["dq"][t + 1:150]])
        assert torch.equal(rest, torch.cat([clean["dq"][:t], clean["dq"][t + 1:150]]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_sequences_stay_as_they_are(dtype):
    """A padded batch: the rows behind the last sequence hold NaN and are neither read nor written."""
    c = lc.make([70, 130, 56], 1, 2, 64, 32, dtype, 59)
    want = run_forward(c), run_backward(c)
    T = sum(c["lengths"])
    pad = dict(c)
    for n in ("q", "k", "v", "do"):
        pad[n] = np.concatenate([c[n], np.full((50, *c[n].shape[1:]), np.nan)])
    pad["g"] = np.concatenate([c["g"], np.full((50, 2), np.nan)])
    got = run_forward(pad, uniform=False), run_backward(pad, uniform=False)
    for g, w in zip(got, want):
        for n in g:
            if n in ("final", "d_initial"):
                assert torch.equal(g[n], w[n]), n
            else:
                ref = lc.references(c)
                lc.check(c, n, g[n][:T], ref[0][n], ref[1][n], dtype if n != "dg" else "f32")
                assert bool(g[n][T:].isnan().all()), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_indices(dtype):
    """A state index outside the pool: zero outputs, untouched states, a flag; the other sequences as ever."""
    c = lc.make([40, 60, 30], 1, 2, 32, 32, dtype, 61)
    refs = lc.references(c)
    for bad in (-1, 5, 1 << 30):
        q, k, v, g = _inputs(c)
        o = torch.full((130, 2, 32), float("nan"), dtype=lc.TYPES[dtype], device="cuda")
        start, _ = lc.pool(None, 3, (2, 32, 32), 3)
        start[:3] = lc.f32(c["initial"])
        final = torch.full_like(start, 7.0)
        rows = torch.tensor([0, bad, 2], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_linear_attention(q, k, v, g, o, initial_state=start, final_state=final, state_indices=rows, err_flags=err,
                                 cu_seqlens=lc.cu(c["lengths"]), workspace=_workspace(c, False, False))
        assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
        assert bool((o[40:100] == 0).all()) and bool((final[1] == 7.0).all()) and bool((final[3:] == 7.0).all())
        for s, at in ((0, slice(0, 40)), (2, slice(100, 130))):
            lc.check(c, "o", o[at], refs[0]["o"][at], refs[1]["o"][at], dtype)
            lc.check(c, "final", final[s], refs[0]["final"][s], refs[1]["final"][s])
        do, end = lc.put(c["do"], dtype), torch.zeros_like(start)
        end[:3] = lc.f32(c["d_final"])
        grads = {n: torch.full_like(t.contiguous(), float("nan")) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
        d0 = torch.full_like(start, 7.0)
        err.zero_()
        gdn.gdn_linear_attention_backward(q, k, v, g, do, initial_state=start, d_final_state=end, state_indices=rows,
                                          err_flags=err, cu_seqlens=lc.cu(c["lengths"]), d_initial_state=d0,
                                          workspace=_workspace(c, False, True), **grads)
        assert int(err) == gdn.GDN_DEVERR_BAD_INDEX and bool((d0[1] == 7.0).all()) and bool((d0[3:] == 7.0).all())
        for n, t in grads.items():
            assert bool((t[40:100] == 0).all()), n
            for at in (slice(0, 40), slice(100, 130)):
                lc.check(c, n, t[at], refs[0][n][at], refs[1][n][at], dtype if n != "dg" else "f32")


@pytest.mark.parametrize("table,fine", [([0, 40, 20, 130], [0, 2]), ([0, 40, 500, 500], [0]), ([-5, 40, 100, 130], [1, 2])])
def test_bad_tables(table, fine):
    """Borders that decrease or leave the rows: such sequences are skipped with a flag."""
    c = lc.make([130], 1, 1, 32, 32, "bf16", 67, states=False)
    q, k, v, g = _inputs(c)
    o = torch.full((130, 1, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = gdn.linear_attention_workspace(130, 1, 1, 32, 32, sequences=3, uniform=False)
    gdn.gdn_linear_attention(q, k, v, g, o, cu_seqlens=torch.tensor(table, dtype=torch.int32, device="cuda"), workspace=ws, err_flags=err)
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
    for s in fine:
        at = slice(table[s], table[s + 1])
        d = {n: (x[at] if isinstance(x, np.ndarray) else x) for n, x in c.items()} | {"lengths": [table[s + 1] - table[s]]}
        want, mag = lc.forward(d)["o"], lc._magnitudes(d)["o"]
        # rows that another sequence of the table claims too hold either one's outputs
        once = [i for i in range(at.start, at.stop) if sum(table[j] <= i < table[j + 1] for j in fine) == 1]
        local = [i - at.start for i in once]
        lc.check(d, "o", o[once], want[local], mag[local], "bf16")


def test_no_tokens():
    pool = torch.randn(3, 2, 8, 16, device="cuda")
    q, v = torch.empty(0, 1, 16, device="cuda"), torch.empty(0, 2, 8, device="cuda")
    g, out = torch.empty(0, 2, device="cuda"), torch.zeros_like(pool)
    gdn.gdn_linear_attention(q, q, v, g, torch.empty_like(v), sequences=3, initial_state=pool, final_state=out)
    assert torch.equal(out, pool)
    d0 = torch.zeros_like(pool)
    ws = gdn.linear_attention_workspace(0, 1, 2, 16, 8, sequences=3, backward=True, dtype=torch.float32)
    dg = torch.full((2,), 5.0, device="cuda")
    gdn.gdn_linear_attention_backward(q, q, v, torch.zeros(2, device="cuda"), v, sequences=3, d_final_state=pool, d_initial_state=d0,
                                      workspace=ws, dg=dg)
    assert torch.equal(d0, pool) and bool((dg == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_segments(dtype):
    """More sequences than a warp counts at once, among them one of many segments."""
    r = np.random.default_rng(5)
    lengths = [int(n) for n in r.integers(0, 4, size=70)]
    lengths[41] = 900
    c = lc.make(lengths, 1, 1, 16, 8, dtype, 71)
    refs = lc.references(c)
    compare(c, run_forward(c), refs)
    compare(c, run_backward(c), refs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_streams_and_graphs(dtype):
    c = lc.make([300, 210], 1, 2, 64, 64, dtype, 73)
    q, k, v, g = _inputs(c)
    do, o = lc.put(c["do"], dtype), torch.empty(510, 2, 64, dtype=lc.TYPES[dtype], device="cuda")
    grads = {n: torch.empty_like(t.contiguous()) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    kw = {"cu_seqlens": lc.cu(c["lengths"])}
    fwd = gdn.gdn_linear_attention(q, k, v, g, o, workspace=_workspace(c, False, False), prepare=True, **kw)
    bwd = gdn.gdn_linear_attention_backward(q, k, v, g, do, workspace=_workspace(c, False, True), prepare=True, **grads, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fwd(s), bwd(s)
    s.synchronize()
    want = [o.clone()] + [t.clone() for t in grads.values()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd(), bwd()
    for _ in range(2):
        for t in (o, *grads.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o, *grads.values()), want):
            assert torch.equal(a, b)                     # sums are taken in a fixed order
    c["initial"] = c["d_final"] = None
    compare(c, {"o": o, **grads})


# ---- single tokens -----------------------------------------------------------------------------
def run_step(B, H, HV, K, V, dtype, sdt, *, fixed=False, turned=0, interleaved=False, layout="rows", magnitude=1.0, seed=0,
             out="same", indexed=True):
    r = np.random.default_rng(seed)
    c = lc.make([B], H, HV, K, V, dtype, seed, fixed=fixed, states=False)
    slots = r.permutation(B + 3)[:B].astype(np.int32) if indexed else np.arange(B, dtype=np.int32)
    S = lc.values(r.normal(size=(B + 3, HV, V, K)), sdt)
    state = torch.from_numpy(S).to(lc.TYPES[sdt]).cuda()
    q, k, v, g = _inputs(c, layout)
    o = torch.full((B, HV, V), float("nan"), dtype=lc.TYPES[dtype if out == "same" else out], device="cuda")
    pos = r.integers(-100, 1 << 20, size=B).astype(np.int32)
    f = gdn.rotary_frequencies(turned) if turned else None
    kw = {"positions": torch.from_numpy(pos).cuda(), "frequencies": f, "interleaved": interleaved, "magnitude": magnitude} if turned else {}
    before = state.clone()
    gdn.gdn_linear_attention_step(q, k, v, g, state, o, torch.from_numpy(slots).cuda() if indexed else None, **kw)
    torch.cuda.synchronize()
    qq, kk = c["q"], c["k"]
    grow = 1.0
    if turned:
        args = (pos, f.cpu().numpy(), magnitude, interleaved)
        qq, kk, grow = lc.turn(qq, *args), lc.turn(kk, *args), 2.0
    G = HV // H
    a = np.exp(np.broadcast_to(c["g"], (B, HV)))[:, :, None, None]
    wide = lambda x: np.repeat(x, G, 1)
    now = a * S[slots] + c["v"][..., :, None] * wide(kk)[..., None, :]
    size = a * np.abs(S[slots]) + np.abs(c["v"])[..., :, None] * np.maximum(1.0, np.abs(wide(kk)))[..., None, :] * grow
    want, wsize = (np.einsum("bhvk,bhk->bhv", x, np.abs(wide(qq)) * grow + 1e-3 if i else wide(qq)) * c["scale"]
                   for i, x in enumerate((now, size)))
    # K additions, the exponential (2^-22), the angles' cosines and sines (2^-21 of a pair's size) and a few roundings
    u = (K + 32) * 2.0 ** -23
    half = lambda t: torch.finfo(t.dtype).eps / 2
    got = o.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= u * wsize + half(o) * np.abs(want))
    st = state.double().cpu().numpy()
    assert np.all(np.abs(st[slots] - now) <= 2.0 ** -20 * size * 2 + half(state) * np.abs(now) * (1 + 2.0 ** -8))
    rest = np.setdiff1d(np.arange(B + 3), slots)
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("sdt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,HV,K,V", [(1, 1, 1, 16, 1), (3, 2, 4, 32, 33), (2, 16, 32, 128, 128), (40, 4, 8, 64, 100), (5, 1, 3, 128, 300),
                                        (70, 3, 9, 16, 128), (30, 24, 24, 64, 64)])
def test_step(B, H, HV, K, V, dtype, sdt):
    run_step(B, H, HV, K, V, dtype, sdt, seed=B + K, fixed=B % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,turned,interleaved,magnitude", [(16, 16, False, 1.0), (64, 30, True, 1.25), (128, 64, False, 1.0), (128, 128, True, 1.0),
                                                            (32, 2, False, 0.5), (64, 38, False, 1.0)])
def test_step_with_positions(K, turned, interleaved, magnitude, dtype):
    run_step(9, 2, 4, K, 48, dtype, "f32", turned=turned, interleaved=interleaved, magnitude=magnitude, seed=K + turned)


@pytest.mark.parametrize("layout", ["dense", "odd", "heads"])
@pytest.mark.parametrize("turned", [0, 20])
def test_step_layouts(layout, turned):
    run_step(6, 2, 4, 64, 50, "bf16", "f32", turned=turned, layout=layout, seed=3)
    run_step(6, 2, 4, 64, 50, "f32", "bf16", turned=turned, layout=layout, seed=4, out="bf16", indexed=False)


def test_step_skips_pads_and_bad_slots():
    B, HV, V, K = 5, 2, 24, 32
    q, v = torch.randn(B, 1, K, device="cuda"), torch.randn(B, HV, V, device="cuda")
    state, out = torch.randn(4, HV, V, K, device="cuda"), torch.full((B, HV, V), float("nan"), device="cuda")
    before, err = state.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, 0, 9, -3, 1], dtype=torch.int32, device="cuda")
    gdn.gdn_linear_attention_step(q, q, v, torch.zeros(HV, device="cuda"), state, out, idx, pad_slot_id=0, err_flags=err)
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX and bool((out[1:4] == 0).all()) and not bool(out.isnan().any())
    assert torch.equal(state[0], before[0]) and torch.equal(state[3], before[3])
    want = before[2] + v[0][:, :, None] * q[0][:, None, :]
    assert torch.allclose(state[2], want, atol=1e-6) and not torch.equal(state[1], before[1])


# ---- together ----------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_single_tokens(dtype):
    """Ragged prompts with positions, then steps that turn q and k themselves: the outputs of one long prompt."""
    H, HV, K, V, lengths, extra = 2, 4, 64, 48, [130, 5, 0, 64], 6
    full = lc.make([n + extra for n in lengths], H, HV, K, V, dtype, 79, fixed=True, states=False)
    f = gdn.rotary_frequencies(32)
    S, starts = len(lengths), np.concatenate([[0], np.cumsum([n + extra for n in lengths])])
    pos = np.concatenate([np.arange(n + extra) for n in lengths]).astype(np.int32)
    prompt = np.concatenate([starts[s] + np.arange(lengths[s]) for s in range(S)])
    q, k, v = (lc.put(full[n], dtype, "dense") for n in ("q", "k", "v"))
    g = lc.f32(full["g"])
    at = torch.from_numpy(prompt).cuda()
    qp, kp = q[at].contiguous(), k[at].contiguous()
    gdn.gdn_rotary(qp, kp, torch.from_numpy(pos[prompt]).cuda(), f)
    pool, rows = lc.pool(None, S, (HV, V, K), 9)
    pool.zero_()
    o = torch.empty(len(prompt), HV, V, dtype=lc.TYPES[dtype], device="cuda")
    gdn.gdn_linear_attention(qp, kp, v[at].contiguous(), g, o, cu_seqlens=lc.cu(lengths), final_state=pool, state_indices=rows,
                             workspace=gdn.linear_attention_workspace(len(prompt), H, HV, K, V, sequences=S, uniform=False, dtype=o.dtype))
    outs = []
    for i in range(extra):
        now = torch.tensor([starts[s] + lengths[s] + i for s in range(S)], device="cuda")
        out = torch.empty(S, HV, V, dtype=lc.TYPES[dtype], device="cuda")
        gdn.gdn_linear_attention_step(q[now], k[now], v[now], g, pool, out, rows,
                                      positions=torch.from_numpy(pos[now.cpu().numpy()]).cuda(), frequencies=f)
        outs.append(out.double().cpu().numpy())
    turned = dict(full)
    for n in ("q", "k"):
        turned[n] = lc.turn(full[n], pos, f.cpu().numpy())
    want, mag = lc.forward(turned)["o"], lc._magnitudes(turned)["o"]
    # a turned bf16 value is rounded once more before the prompt takes it (both q and k: 2^-8 of a term's size)
    u = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -13) * 2
    assert np.all(np.abs(o.double().cpu().numpy() - want[prompt]) <= u * mag[prompt] + 1e-6)
    for i in range(extra):
        now = [starts[s] + lengths[s] + i for s in range(S)]
        assert np.all(np.abs(outs[i] - want[now]) <= u * mag[now] + 1e-6)
