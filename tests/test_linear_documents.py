"""Linear attention over hundreds and thousands of packed documents: right for each of them, whole and cut ones, with rows between
them that are no one's; and at a time a token that does not grow with their number."""
import numpy as np
import pytest
import torch

import linear_cases as lc
import ssm_recurrent_decode_gb300 as gdn
from test_parity_linear import compare, run_backward, run_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,HV,fixed", [
    ([int(n) for n in np.random.default_rng(1).integers(0, 9, size=700)], 1, 2, False),
    ([3, 0, 1] * 40 + [700] + [5] * 90 + [260, 0, 900], 1, 1, True),      # some of them cut, the last one among them
    ([1] * 65, 2, 2, False),
])
def test_each_document(lengths, H, HV, fixed, dtype):
    c = lc.make(lengths, H, HV, 16, 8, dtype, 7 + len(lengths), fixed=fixed)
    refs = lc.references(c)
    compare(c, run_forward(c, uniform=False), refs)
    compare(c, run_backward(c, uniform=False), refs)


def _packed(S, L, H, HV, K, V, dtype, seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    T = S * L
    x = {"q": n(T, H, K), "k": n(T, H, K), "v": n(T, HV, V), "do": n(T, HV, V),
         "g": -torch.exp(torch.rand(T, HV, generator=gen, device="cuda") * 5.0 - 6.0)}
    space = lambda b: gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, uniform=False, backward=b, dtype=dtype)
    out = {"o": torch.empty_like(x["v"]), "dq": torch.empty_like(x["q"]), "dk": torch.empty_like(x["k"]),
           "dv": torch.empty_like(x["v"]), "dg": torch.empty_like(x["g"])}
    kw = {"cu_seqlens": torch.arange(S + 1, dtype=torch.int32, device="cuda") * L, "prepare": True}
    args = (x["q"], x["k"], x["v"], x["g"])
    fwd = gdn.gdn_linear_attention(*args, out["o"], workspace=space(False), **kw)
    bwd = gdn.gdn_linear_attention_backward(*args, x["do"], workspace=space(True), **kw, **{n: t for n, t in out.items() if n != "o"})
    return x, out, fwd, bwd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_thousand_documents_of_several_chunks(dtype):
    """The first, a middle and the last of 2000 documents of 150 tokens are what calls of their own give."""
    S, L, H, HV, K, V = 2000, 150, 1, 2, 32, 32
    x, out, fwd, bwd = _packed(S, L, H, HV, K, V, dtype)
    fwd(), bwd()
    torch.cuda.synchronize()
    name = {torch.bfloat16: "bf16", torch.float32: "f32"}[dtype]
    for s in (0, 1, 777, 1998, 1999):
        at = slice(s * L, s * L + L)
        c = {n: t[at].double().cpu().numpy() for n, t in x.items()}
        c |= {"initial": None, "d_final": None, "lengths": [L], "scale": K ** -0.5, "dtype": name}
        ref, mag = lc.references(c)
        for n, t in out.items():
            lc.check(c, n, t[at], ref[n], mag[n], name if n != "dg" else "f32")


def test_a_table_of_many_with_borders_that_decrease():
    """Hundreds of sequences that claim the same rows again and again: nothing behind the workspace is touched, the flag is
    raised, and the first one has its outputs."""
    from test_linear_machine import Guarded, _random
    T, H, HV, K, V = 2000, 2, 4, 64, 32
    x = _random(1, T, H, HV, K, V, "bf16", 61)
    table = torch.tensor([0, T] + [0, T] * 150, dtype=torch.int32, device="cuda")
    S, guards = len(table) - 1, []

    def space(backward):
        ws = gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, uniform=False, backward=backward)
        guards.append(Guarded(ws.fill_(0xFF)))
        return guards[-1].t

    err, o = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(x["v"])
    args = (x["q"], x["k"], x["v"], x["g"])
    gdn.gdn_linear_attention(*args, o, cu_seqlens=table, workspace=space(False), err_flags=err)
    grads = {n: torch.empty_like(x[i]) for n, i in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    gdn.gdn_linear_attention_backward(*args, x["do"], cu_seqlens=table, workspace=space(True), **grads)
    torch.cuda.synchronize()
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
    assert all(g.intact() for g in guards)
    d = lambda t: t.double().cpu().numpy()
    c = {"q": d(x["q"]), "k": d(x["k"]), "v": d(x["v"]), "do": d(x["do"]), "g": d(x["g"]), "initial": None, "d_final": None,
         "lengths": [T], "scale": K ** -0.5, "dtype": "bf16"}
    lc.check(c, "o", o, lc.forward(c)["o"], lc._magnitudes(c)["o"], "bf16")


def test_time_does_not_grow_with_their_number():
    """Gradients of 1024 documents take less than four times as long a token as those of 64 (it was eleven times when
    every one's CTAs looked through all of them; about once is expected)."""
    def per_token(S):
        x, out, fwd, bwd = _packed(S, 256, 16, 32, 64, 64, torch.bfloat16)
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            bwd()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times) / x["q"].shape[0]

    assert per_token(1024) < 4.0 * per_token(64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_in_place_and_bad_indices_among_many(dtype):
    """A pool read and written in place by a hundred sequences, some cut, some empty; two with an index outside the pool have zero
    outputs and gradients and touch no state, the others are right."""
    lengths = [4, 0, 300, 1] * 25
    S, H, HV, K, V = len(lengths), 1, 2, 32, 24
    c = lc.make(lengths, H, HV, K, V, dtype, 31)
    refs = lc.references(c)
    T, bad = sum(lengths), (6, 99)
    start, rows = lc.pool(c["initial"], S, (HV, V, K), 3)
    end, _ = lc.pool(c["d_final"], S, (HV, V, K), 3)
    keep = start.clone()
    slots = rows.clone()
    slots[bad[0]], slots[bad[1]] = -7, S + 2
    q, k, v, do = (lc.put(c[n], dtype, "dense") for n in ("q", "k", "v", "do"))
    g, err = lc.f32(c["g"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    space = lambda b: gdn.linear_attention_workspace(T, H, HV, K, V, sequences=S, uniform=False, backward=b, dtype=lc.TYPES[dtype]).fill_(0xFF)
    grads = {n: torch.full_like(t, float("nan")) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    o, d0 = torch.full_like(v, float("nan")), torch.full_like(start, 7.0)
    kw = {"cu_seqlens": lc.cu(lengths), "state_indices": slots, "initial_state": start}
    gdn.gdn_linear_attention_backward(q, k, v, g, do, d_final_state=end, d_initial_state=d0, err_flags=err, workspace=space(True), **kw, **grads)
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
    err.zero_()
    gdn.gdn_linear_attention(q, k, v, g, o, final_state=start, err_flags=err, workspace=space(False), **kw)
    torch.cuda.synchronize()
    assert int(err) == gdn.GDN_DEVERR_BAD_INDEX
    ends = np.cumsum(lengths)
    lost = np.zeros(T, dtype=bool)
    for s in bad:
        lost[ends[s] - lengths[s]:ends[s]] = True
    good = [s for s in range(S) if s not in bad]
    for n, t in {"o": o, **grads}.items():
        assert bool((t[torch.from_numpy(lost).cuda()] == 0).all()), n
        at = torch.from_numpy(~lost).cuda()
        lc.check(c, n, t[at], refs[0][n][~lost], refs[1][n][~lost], dtype if n != "dg" else "f32")
    used = rows[good].long()
    for n, p in (("final", start), ("d_initial", d0)):
        lc.check(c, n, p[used], refs[0][n][good], refs[1][n][good])
    rest = [i for i in range(S + 2) if i not in used.tolist()]
    assert torch.equal(start[rest], keep[rest]) and bool((d0[rest] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_debug_build_agrees_over_many(dtype):
    """Its kernels check the segments, rows, chunks and workspace entries that they compute; the bits are the same."""
    lengths = [5, 0, 290, 1, 130] * 20
    c = lc.make(lengths, 2, 4, 64, 40, dtype, 37)
    runs = []
    for debug in (False, True):
        def both(c=c):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = run_forward(c, uniform=False, err=err) | run_backward(c, uniform=False, err=err)
            assert int(err) == 0
            return out
        if debug:
            with gdn.using_debug_build():
                runs.append(both())
        else:
            runs.append(both())
    for n, t in runs[0].items():
        assert torch.equal(t, runs[1][n]), n
