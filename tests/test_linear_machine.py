"""Linear attention and rotary positions at sizes that fill the GPU: repeated calls give the same bits, heads of large calls
and sequences of many segments agree with the 64-bit references, calls on two streams do not touch each other's
workspaces, a run of a prompt and the tokens behind it is one attention, and guard bands around everything that is
written stay as they were."""
import numpy as np
import pytest
import torch

import linear_cases as lc
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _random(S, L, H, HV, K, V, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(lc.TYPES[dtype])
    T = S * L
    g = -torch.exp(torch.rand(T, HV, generator=gen, device="cuda") * 5.0 - 6.0)
    f = lambda: torch.randn(S, HV, V, K, generator=gen, device="cuda")
    return {"q": n(T, H, K), "k": n(T, H, K), "v": n(T, HV, V), "do": n(T, HV, V), "g": g, "initial": f(), "d_final": f()}


def _calls(x, S, dtype):
    T, H, K = x["q"].shape
    HV, V = x["v"].shape[1:]
    nan = lambda t: torch.full_like(t, float("nan"))
    o, final, err = nan(x["v"]), nan(x["initial"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = {"dq": nan(x["q"]), "dk": nan(x["k"]), "dv": nan(x["v"]), "dg": nan(x["g"]), "d_initial_state": nan(x["initial"])}
    space = lambda b: gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, backward=b, dtype=lc.TYPES[dtype])
    args = (x["q"], x["k"], x["v"], x["g"])
    kw = {"sequences": S, "initial_state": x["initial"], "err_flags": err, "prepare": True}
    fwd = gdn.gdn_linear_attention(*args, o, final_state=final, workspace=space(False), **kw)
    bwd = gdn.gdn_linear_attention_backward(*args, x["do"], d_final_state=x["d_final"], workspace=space(True), **kw, **grads)
    return fwd, bwd, {"o": o, "final": final, **grads}, err


def _check_heads(x, S, L, out, dtype, sequences, heads):
    """Some sequences and q/k heads of a large call against the references."""
    H, HV = x["q"].shape[1], x["v"].shape[1]
    G, K = HV // H, x["q"].shape[2]
    for s in sequences:
        for h in heads:
            rows, hv = slice(s * L, (s + 1) * L), slice(h * G, (h + 1) * G)
            d = lambda t: t.double().cpu().numpy()
            c = {"q": d(x["q"][rows, h:h + 1]), "k": d(x["k"][rows, h:h + 1]), "v": d(x["v"][rows, hv]), "do": d(x["do"][rows, hv]),
                 "g": d(x["g"][rows, hv]), "initial": d(x["initial"][s:s + 1, hv]), "d_final": d(x["d_final"][s:s + 1, hv]),
                 "lengths": [L], "scale": K ** -0.5, "dtype": dtype}
            ref, mag = lc.references(c)
            got = {"o": out["o"][rows, hv], "final": out["final"][s:s + 1, hv], "dq": out["dq"][rows, h:h + 1],
                   "dk": out["dk"][rows, h:h + 1], "dv": out["dv"][rows, hv], "dg": out["dg"][rows, hv],
                   "d_initial": out["d_initial_state"][s:s + 1, hv]}
            for n, t in got.items():
                lc.check(c, n, t, ref[n], mag[n], dtype if n in ("o", "dq", "dk", "dv") else "f32")


@pytest.mark.parametrize("dtype,S,L,H,HV,K,V,repeats", [
    ("bf16", 8, 384, 32, 32, 128, 128, 12),       # more CTAs than SMs, whole sequences
    ("bf16", 1, 4096, 4, 4, 128, 128, 12),        # one sequence in many segments
    ("bf16", 2, 1500, 6, 18, 64, 128, 8),         # shared heads, segments with a ragged end
    ("bf16", 5, 640, 16, 32, 128, 100, 8),        # a value size that is no multiple of eight
    ("bf16", 3, 900, 12, 24, 128, 61, 8),         # rows that are not 16-byte aligned
    ("f32", 2, 700, 8, 16, 128, 128, 6),
    ("f32", 1, 3000, 2, 2, 64, 64, 6),
])
def test_large_calls_repeat_and_agree(dtype, S, L, H, HV, K, V, repeats):
    x = _random(S, L, H, HV, K, V, dtype, 100 + L)
    fwd, bwd, out, err = _calls(x, S, dtype)
    fwd(), bwd()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in out.items()}
    _check_heads(x, S, L, want, dtype, (S - 1,), (0, H - 1))
    for _ in range(repeats):
        for t in out.values():
            t.fill_(float("nan"))
        fwd(), bwd()
    torch.cuda.synchronize()
    for n, t in out.items():
        assert torch.equal(t, want[n]), n
    assert int(err) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    S, L = 2, 1100
    xs = [_random(S, L, 8, 8, 64, 64, dtype, 7 + i) for i in range(2)]
    calls = [_calls(x, S, dtype) for x in xs]
    torch.cuda.synchronize()
    want = []
    for fwd, bwd, out, _ in calls:
        fwd(), bwd()
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in out.items()})
        for t in out.values():
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(4):
        for s, (fwd, bwd, _, _) in zip(streams, calls):
            fwd(s), bwd(s)
    torch.cuda.synchronize()
    for w, (_, _, out, err) in zip(want, calls):
        assert int(err) == 0
        for n, t in out.items():
            assert torch.equal(t, w[n]), n


def _pair_lengths(x, turned, interleaved):
    n, out = turned // 2, np.abs(x)
    a, b = (slice(0, turned, 2), slice(1, turned, 2)) if interleaved else (slice(0, n), slice(n, turned))
    out[..., a] = out[..., b] = np.hypot(x[..., a], x[..., b])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_prompt_and_the_tokens_behind_it(dtype, interleaved):
    """rotary, attention over prompts into the slots of a pool, single tokens from those slots: the outputs and states of one
    attention over all tokens with turned q and k."""
    lengths, more, H, HV, K, V, turned = [130, 1, 300], 5, 2, 4, 64, 48, 40
    S = len(lengths)
    full = lc.make([n + more for n in lengths], H, HV, K, V, dtype, 97, states=False)
    ends = np.cumsum([n + more for n in lengths])
    prompt = np.concatenate([np.arange(e - n - more, e - more) for e, n in zip(ends, lengths)])
    position = np.concatenate([np.arange(n + more) for n in lengths]).astype(np.int32)
    f = gdn.rotary_frequencies(turned)
    put = lambda n, rows: lc.put(full[n][rows], dtype, "dense")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool = torch.full((6, HV, V, K), 7.0, device="cuda")
    start = torch.zeros_like(pool)
    q, k, v = put("q", prompt), put("k", prompt), put("v", prompt)
    gdn.gdn_rotary(q, k, torch.from_numpy(position[prompt]).cuda(), f, interleaved=interleaved)
    o = torch.empty_like(v)
    ws = gdn.linear_attention_workspace(len(prompt), H, HV, K, V, sequences=S, uniform=False, dtype=lc.TYPES[dtype])
    gdn.gdn_linear_attention(q, k, v, lc.f32(full["g"][prompt]), o, cu_seqlens=lc.cu(lengths), state_indices=slots,
                             initial_state=start, final_state=pool, workspace=ws)
    got = np.zeros((len(position), HV, V))
    got[prompt] = o.double().cpu().numpy()
    for i in range(more):
        rows = ends - more + i
        step_o = torch.empty(S, HV, V, dtype=lc.TYPES[dtype], device="cuda")
        gdn.gdn_linear_attention_step(put("q", rows), put("k", rows), put("v", rows), lc.f32(full["g"][rows]), pool, step_o, slots,
                                      positions=torch.from_numpy(position[rows]).cuda(), frequencies=f, interleaved=interleaved)
        got[rows] = step_o.double().cpu().numpy()
    torch.cuda.synchronize()
    # the prompt's q and k are rounded to the type after they are turned (half a step each), a token's are not
    args = (position, f.cpu().numpy(), 1.0, interleaved)
    turnt = dict(full, q=lc.turn(full["q"], *args), k=lc.turn(full["k"], *args))
    want = lc.forward(turnt)
    half = torch.finfo(lc.TYPES[dtype]).eps / 2
    # a turned channel is at most its pair's length, and its rounding half a step of that
    wide = dict(full, q=_pair_lengths(full["q"], turned, interleaved), k=_pair_lengths(full["k"], turned, interleaved))
    mag = lc._magnitudes(wide)
    L = max(full["lengths"])
    u = (L + K + V + 64) * 2.0 ** -23 + (2 * half + 2.0 ** -8 if dtype == "bf16" else 2 * half)
    assert np.all(np.abs(got - want["o"]) <= u * mag["o"] * (1 + half) + half * np.abs(want["o"]))
    now = pool[slots.long()].double().cpu().numpy()
    assert np.all(np.abs(now - want["final"]) <= ((L + 64) * 2.0 ** -23 + half) * mag["final"])
    assert bool((pool[[1, 3, 5]] == 7.0).all())


GUARD = 4096


class Guarded:
    def __init__(self, src):
        self.n = src.numel() * src.element_size()
        self.raw = torch.full((2 * GUARD + self.n,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + self.n].view(src.dtype).view(src.shape)
        self.t.copy_(src)

    def intact(self):
        return bool((self.raw[:GUARD] == 0xA5).all()) and bool((self.raw[GUARD + self.n:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,HV,K,V", [([300, 1, 129], 1, 2, 64, 50), ([128], 2, 2, 128, 128), ([700, 0, 20], 1, 1, 16, 7),
                                               ([45, 260], 3, 3, 128, 96)])
def test_only_its_buffers_are_written(lengths, H, HV, K, V, dtype):
    c = lc.make(lengths, H, HV, K, V, dtype, 300 + V)
    T, S = sum(lengths), len(lengths)
    q, k, v, do = (lc.put(c[n], dtype, "dense") for n in ("q", "k", "v", "do"))
    g, initial, d_final = lc.f32(c["g"]), lc.f32(c["initial"]), lc.f32(c["d_final"])
    b = {}

    def guard(name, like):
        b[name] = Guarded(like)
        return b[name].t

    kw = {"cu_seqlens": lc.cu(lengths), "initial_state": initial}

    def space(name, backward):
        ws = gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, uniform=False, backward=backward, dtype=lc.TYPES[dtype])
        return ws if ws is None else guard(name, ws.fill_(0xFF))

    gdn.gdn_linear_attention(q, k, v, g, guard("o", v), final_state=guard("final", initial), workspace=space("w1", False), **kw)
    gdn.gdn_linear_attention_backward(q, k, v, g, do, dq=guard("dq", q), dk=guard("dk", k), dv=guard("dv", v), dg=guard("dg", g),
                                      d_final_state=d_final, d_initial_state=guard("d0", initial), workspace=space("w2", True), **kw)
    n = min(T, 9)
    pool = guard("pool", torch.zeros(n, HV, V, K, device="cuda"))
    gdn.gdn_linear_attention_step(q[:n], k[:n], v[:n], g[:n].contiguous(), pool, guard("step", v[:n]))
    gdn.gdn_rotary(q, k, torch.arange(T, dtype=torch.int32, device="cuda"), gdn.rotary_frequencies(K // 2),
                   q_out=guard("q2", q), k_out=guard("k2", k))
    torch.cuda.synchronize()
    for name, x in b.items():
        assert x.intact(), name
    ref, mag = lc.references(c)
    for name, key in (("o", "o"), ("final", "final"), ("dq", "dq"), ("dk", "dk"), ("dv", "dv"), ("dg", "dg"), ("d0", "d_initial")):
        lc.check(c, key, b[name].t, ref[key], mag[key], dtype if name in ("o", "dq", "dk", "dv") else "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,L,H,HV,K,V", [(3, 333, 2, 4, 64, 50), (2, 128, 1, 1, 128, 128), (1, 1100, 2, 2, 16, 9)])
def test_the_debug_build_agrees(S, L, H, HV, K, V, dtype):
    """Its kernels check the indices that they compute: none may be out of range, and the bits are the same."""
    x = _random(S, L, H, HV, K, V, dtype, 500 + L)
    results = []
    for debug in (False, True):
        def run():
            fwd, bwd, out, err = _calls(x, S, dtype)
            fwd(), bwd()
            pool, o = x["initial"].clone(), torch.empty_like(x["v"][:S])
            positions = torch.arange(S * L, dtype=torch.int32, device="cuda")
            table = gdn.rotary_frequencies(K // 2)
            gdn.gdn_linear_attention_step(x["q"][:S], x["k"][:S], x["v"][:S], x["g"][:S], pool, o, positions=positions[:S],
                                          frequencies=table, err_flags=err)
            q, k = x["q"].clone(), x["k"].clone()
            gdn.gdn_rotary(q, k, positions, table)
            torch.cuda.synchronize()
            assert int(err) == 0
            return list(out.values()) + [pool, o, q, k]

        if debug:
            with gdn.using_debug_build():
                results.append(run())
        else:
            results.append(run())
    for a, b in zip(*results):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("repeat", [1, 2, 40])
def test_a_table_that_claims_rows_again_and_again(repeat, dtype):
    """Borders that decrease can name more segments than the workspace has room for: nothing behind it is touched, the flag is
    raised, and the first sequence, which is in order, has its outputs."""
    T, H, HV, K, V = 2000, 2, 4, 64, 32
    x = _random(1, T, H, HV, K, V, dtype, 61)
    table = torch.tensor([0, T] + [0, T] * repeat, dtype=torch.int32, device="cuda")
    S = len(table) - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    guards = []

    def space(backward):
        ws = gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, uniform=False, backward=backward, dtype=lc.TYPES[dtype])
        guards.append(Guarded(ws.fill_(0xFF)))
        return guards[-1].t

    o = torch.empty_like(x["v"])
    args = (x["q"], x["k"], x["v"], x["g"])
    gdn.gdn_linear_attention(*args, o, cu_seqlens=table, workspace=space(False), err_flags=err)
    grads = {n: torch.empty_like(x[i]) for n, i in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    gdn.gdn_linear_attention_backward(*args, x["do"], cu_seqlens=table, workspace=space(True), **grads)
    torch.cuda.synchronize()
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
    assert all(g.intact() for g in guards)
    d = lambda t: t.double().cpu().numpy()
    c = {"q": d(x["q"]), "k": d(x["k"]), "v": d(x["v"]), "do": d(x["do"]), "g": d(x["g"]), "initial": None, "d_final": None,
         "lengths": [T], "scale": K ** -0.5, "dtype": dtype}
    lc.check(c, "o", o, lc.forward(c)["o"], lc._magnitudes(c)["o"], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_broadcast_inputs(dtype):
    """Strides of zero: one q for all heads, one v for all tokens."""
    c = lc.make([200, 90], 2, 4, 32, 40, dtype, 88, states=False)
    c["q"] = np.broadcast_to(c["q"][:, :1], c["q"].shape).copy()
    c["v"] = np.broadcast_to(c["v"][:1], c["v"].shape).copy()
    q = lc.put(c["q"][:, :1], dtype, "dense").expand(-1, 2, -1)
    v = lc.put(c["v"][:1], dtype, "dense").expand(290, -1, -1)
    k, do, g = lc.put(c["k"], dtype, "dense"), lc.put(c["do"], dtype, "dense"), lc.f32(c["g"])
    space = lambda b: gdn.linear_attention_workspace(290, 2, 4, 32, 40, sequences=2, uniform=False, backward=b, dtype=lc.TYPES[dtype])
    full = lambda t: torch.full_like(t.contiguous(), float("nan"))
    o, grads = full(v), {"dq": full(q), "dk": full(k), "dv": full(v), "dg": full(g)}
    gdn.gdn_linear_attention(q, k, v, g, o, cu_seqlens=lc.cu(c["lengths"]), workspace=space(False))
    gdn.gdn_linear_attention_backward(q, k, v, g, do, cu_seqlens=lc.cu(c["lengths"]), workspace=space(True), **grads)
    torch.cuda.synchronize()
    ref, mag = lc.references(c)
    for n, t in {"o": o, **grads}.items():
        lc.check(c, n, t, ref[n], mag[n], dtype if n != "dg" else "f32")


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 72), (16, 24)])
def test_rows_at_any_address(K, V, offset):
    """bf16 rows that start 2, 4, 8 or 16 bytes past their alignment, at strides that keep them there."""
    c = lc.make([140, 75], 2, 4, K, V, "bf16", 90 + offset)
    T, H, HV = 215, 2, 4

    def put(a):
        heads, n = a.shape[1:]
        rows = torch.full((T, offset + heads * n), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = rows[:, offset:].unflatten(1, (heads, n))
        view.copy_(torch.from_numpy(a))
        return view

    q, k, v, do, g = put(c["q"]), put(c["k"]), put(c["v"]), put(c["do"]), lc.f32(c["g"])
    o, grads = torch.empty_like(v), {"dq": put(c["q"]), "dk": put(c["k"]), "dv": put(c["v"]), "dg": torch.empty_like(g)}
    space = lambda b: gdn.linear_attention_workspace(T, H, HV, K, V, sequences=2, uniform=False, backward=b)
    start, end = lc.f32(c["initial"]), lc.f32(c["d_final"])
    final, d0 = torch.empty_like(start), torch.empty_like(start)
    gdn.gdn_linear_attention(q, k, v, g, o, initial_state=start, final_state=final, cu_seqlens=lc.cu(c["lengths"]), workspace=space(False))
    gdn.gdn_linear_attention_backward(q, k, v, g, do, initial_state=start, d_final_state=end, d_initial_state=d0,
                                      cu_seqlens=lc.cu(c["lengths"]), workspace=space(True), **grads)
    torch.cuda.synchronize()
    ref, mag = lc.references(c)
    for n, t in {"o": o, "final": final, "d_initial": d0, **grads}.items():
        lc.check(c, n, t, ref[n], mag[n], "bf16" if n in ("o", "dq", "dk", "dv") else "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_and_states_gigabytes_apart(dtype):
    """Offsets beyond 32 bits: token rows 2^30 elements apart, and the last slots of a pool of 9 GB."""
    T, H, HV, K, V = 5, 2, 4, 128, 128
    c = lc.make([T], H, HV, K, V, dtype, 77)
    c["d_final"] = None
    gap = 1 << 30
    memory = torch.empty((T - 1) * gap + 16384, dtype=lc.TYPES[dtype], device="cuda")
    used = [0]

    def far(a=None, heads=None, n=None):
        heads, n = (a.shape[1], a.shape[2]) if a is not None else (heads, n)
        t = memory[used[0]:].as_strided((T, heads, n), (gap, n, 1))
        used[0] += heads * n
        if a is not None:
            t.copy_(torch.from_numpy(np.ascontiguousarray(a)))
        return t

    q, k, v, do = (far(c[n]) for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = far(None, HV, V), far(None, H, K), far(None, H, K), far(None, HV, V)
    g = lc.f32(c["g"])
    slots, num = torch.tensor([4290], dtype=torch.int32, device="cuda"), 4300
    pool = torch.empty(num, HV, V, K, device="cuda")
    pool[4290] = lc.f32(c["initial"][0])
    gdn.gdn_linear_attention(q, k, v, g, o, sequences=1, state_indices=slots, initial_state=pool, final_state=pool)
    final = pool[4290:4291].clone()
    pool[4290] = lc.f32(c["initial"][0])
    dg = torch.empty_like(g)
    ws = gdn.linear_attention_workspace(T, H, HV, K, V, backward=True, dtype=lc.TYPES[dtype])
    gdn.gdn_linear_attention_backward(q, k, v, g, do, sequences=1, state_indices=slots, initial_state=pool, dq=dq, dk=dk, dv=dv, dg=dg,
                                      workspace=ws)
    torch.cuda.synchronize()
    ref, mag = lc.references(c)
    for n, t in {"o": o, "final": final, "dq": dq, "dk": dk, "dv": dv, "dg": dg}.items():
        lc.check(c, n, t, ref[n], mag[n], dtype if n in ("o", "dq", "dk", "dv") else "f32")
    # rotary positions there and on dense copies
    near, positions, table = q.contiguous(), torch.arange(T, dtype=torch.int32, device="cuda"), gdn.rotary_frequencies(K)
    gdn.gdn_rotary(q, None, positions, table)
    gdn.gdn_rotary(near, None, positions, table)
    assert torch.equal(q, near)
    del memory, q, k, v, do, o, dq, dk, dv, pool
    # a pool of more than 2^31 entries: the last slot gives what a slot of a small pool gives
    HV = 33
    big, small = torch.empty(4300, HV, V, K, device="cuda"), torch.randn(1, HV, V, K, device="cuda")
    big[4290] = small[0]
    x = [torch.randn(1, n, K, device="cuda").to(lc.TYPES[dtype]) for n in (HV, HV, HV)]
    decay, idx = -torch.rand(1, HV, device="cuda"), torch.tensor([4290], dtype=torch.int32, device="cuda")
    outs = [torch.empty(1, HV, V, device="cuda") for _ in range(2)]
    gdn.gdn_linear_attention_step(*x, decay, big, outs[0], idx)
    gdn.gdn_linear_attention_step(*x, decay, small, outs[1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(big[4290], small[0])
    gdn.gdn_linear_attention(*x, decay, outs[0], sequences=1, state_indices=idx, initial_state=big, final_state=big)
    gdn.gdn_linear_attention(*x, decay, outs[1], sequences=1, initial_state=small, final_state=small)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(big[4290], small[0])
