"""Inputs, 64-bit references and error bounds of the linear-attention and rotary tests.

The bounds are derived from the arithmetic. Every output is a sum of products of inputs and decays; with each factor
replaced by its magnitude the reference gives the sum of the terms' magnitudes, `mag`. After L tokens a term has been
through at most L additions into the state, K or V into an output, and a few factors (a decay's power of two, its
scale, the split of a segment), each with an error of at most 2^-23: (L + K + V + 32) 2^-23 mag. With bf16 inputs a
term of a token's output goes into a matrix product as a score times decays or as part of a state, rounded to bf16 once
for bf16 outputs, at most 2^-8 of it: 2^-8 mag. For fp32 outputs and for dg both are kept as two bf16 numbers, whose
remainder is at most 2^-16 of the term; final states keep 24 bits. dg is the difference of two sums over the tokens
behind it, and its `mag` the sum of their magnitudes. An output of a narrower type adds half a step of it."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def values(a, dtype):
    """fp64 values that `dtype` holds."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).double().numpy()


def make(lengths, H, HV, K, V, dtype, seed, *, fixed=False, states=True, decay=(1e-3, 1.0)):
    r = np.random.default_rng(seed)
    T, S = sum(lengths), len(lengths)
    n = lambda *s: values(r.normal(size=s), dtype)
    g = -np.exp(r.uniform(np.log(decay[0]), np.log(decay[1]), size=HV if fixed else (T, HV)))
    f = lambda a: a.astype(np.float32).astype(np.float64)
    return {"q": n(T, H, K), "k": n(T, H, K), "v": n(T, HV, V), "do": n(T, HV, V), "g": f(g), "lengths": list(lengths),
            "initial": f(r.normal(size=(S, HV, V, K))) if states else None,
            "d_final": f(r.normal(size=(S, HV, V, K))) if states else None, "scale": K ** -0.5, "dtype": dtype}


def forward(c):
    """o [T, HV, V] and final states [S, HV, V, K], token by token."""
    q, k, v = c["q"], c["k"], c["v"]
    T, HV, V = v.shape
    G, K = HV // q.shape[1], q.shape[2]
    a = np.exp(np.broadcast_to(c["g"], (T, HV)))
    o, final = np.zeros((T, HV, V)), np.zeros((len(c["lengths"]), HV, V, K))
    at = 0
    for s, n in enumerate(c["lengths"]):
        S = np.zeros((HV, V, K)) if c["initial"] is None else c["initial"][s].copy()
        for t in range(at, at + n):
            S = a[t][:, None, None] * S + v[t][:, :, None] * np.repeat(k[t], G, 0)[:, None, :]
            o[t] = c["scale"] * np.einsum("hvk,hk->hv", S, np.repeat(q[t], G, 0))
        final[s] = S
        at += n
    return {"o": o, "final": final}


def backward(c):
    """All gradients by the recurrences of their definition; dg_t = exp(g_t) <D_t, S_{t-1}>."""
    q, k, v, do, sc = c["q"], c["k"], c["v"], c["do"], c["scale"]
    T, HV, V = v.shape
    H, K = q.shape[1:]
    G = HV // H
    a = np.exp(np.broadcast_to(c["g"], (T, HV)))
    wide = lambda x: np.repeat(x, G, 0)
    dq, dk, dv, dg = np.zeros((T, HV, K)), np.zeros((T, HV, K)), np.zeros((T, HV, V)), np.zeros((T, HV))
    d0 = np.zeros((len(c["lengths"]), HV, V, K))
    at = 0
    for s, n in enumerate(c["lengths"]):
        S = np.zeros((HV, V, K)) if c["initial"] is None else c["initial"][s].copy()
        before = []
        for t in range(at, at + n):
            before.append(S)
            S = a[t][:, None, None] * S + v[t][:, :, None] * wide(k[t])[:, None, :]
            dq[t] = sc * np.einsum("hvk,hv->hk", S, do[t])
        D = np.zeros((HV, V, K)) if c["d_final"] is None else c["d_final"][s].copy()
        for t in range(at + n - 1, at - 1, -1):
            D = D + sc * do[t][:, :, None] * wide(q[t])[:, None, :]
            dk[t] = np.einsum("hvk,hv->hk", D, v[t])
            dv[t] = np.einsum("hvk,hk->hv", D, wide(k[t]))
            dg[t] = a[t] * (D * before[t - at]).sum((1, 2))
            D = a[t][:, None, None] * D
        d0[s] = D
        at += n
    fold = lambda x: x.reshape(T, H, G, K).sum(2)
    return {"dq": fold(dq), "dk": fold(dk), "dv": dv, "dg": dg.sum(0) if c["g"].ndim == 1 else dg, "d_initial": d0,
            "dq_heads": dq, "dk_heads": dk}


def _magnitudes(c):
    m = {k: np.abs(x) if isinstance(x, np.ndarray) and k != "g" else x for k, x in c.items()}
    f, b = forward(m), backward(m)
    T, HV, _ = c["v"].shape
    wide = lambda x: np.repeat(x, HV // c["q"].shape[1], 1)
    terms = (wide(m["q"]) * b["dq_heads"]).sum(-1) + (wide(m["k"]) * b["dk_heads"]).sum(-1)
    dg, at = np.zeros((T, HV)), 0
    for s, n in enumerate(c["lengths"]):
        end = 0.0 if c["d_final"] is None else (m["d_final"][s] * f["final"][s]).sum((1, 2))
        dg[at:at + n] = terms[at:at + n][::-1].cumsum(0)[::-1] + end
        at += n
    b["dg"] = dg.sum(0) if c["g"].ndim == 1 else dg
    return f | b


def references(c):
    return forward(c) | backward(c), _magnitudes(c)


def check(c, name, got, ref, mag, out=None):
    """|got - ref| within the bound of the module's text."""
    K, V, L = c["q"].shape[2], c["v"].shape[2], max(c["lengths"], default=0)
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    u = (L + K + V + 32) * 2.0 ** -23
    if c["dtype"] == "bf16" and name not in ("final", "d_initial"):
        u += 2.0 ** (-8 if out == "bf16" else -16)
    half = torch.finfo(TYPES[out or "f32"]).eps / 2
    tol = u * mag * (1 + half) + half * np.abs(ref) + 1e-37
    assert np.all(np.isfinite(got)), name
    off = np.abs(got - ref)
    assert np.all(off <= tol), (name, float(np.max(off / tol)), np.unravel_index(np.argmax(off / tol), off.shape))


# ---- tensors -----------------------------------------------------------------------------------
def put(a, dtype, layout="rows"):
    """A device tensor [T, heads, n] of a's values. rows: parts of wider 16-byte rows; odd: rows at odd offsets and
    strides; heads: memory [heads, T, n]."""
    v = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype]).cuda()
    if layout == "dense":
        return v
    T, h, n = v.shape
    nan = float("nan")
    if layout == "rows":
        wide = torch.full((T, h + 1, n), nan, dtype=v.dtype, device="cuda")
        wide[:, :h] = v
        return wide[:, :h]
    if layout == "odd":
        wide = torch.full((T + 1, h * n + 5), nan, dtype=v.dtype, device="cuda")
        view = wide[:T, 3:3 + h * n].unflatten(1, (h, n))
        view.copy_(v)
        return view
    wide = torch.full((h, T + 2, n), nan, dtype=v.dtype, device="cuda")
    view = wide[:, 1:T + 1].transpose(0, 1)
    view.copy_(v)
    return view


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).float().cuda()


def cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def pool(states, S, shape, seed):
    """A pool [S + 2, ...] holding `states` at permuted rows, 7 elsewhere; and the rows."""
    rows = np.random.default_rng(seed).permutation(S + 2)[:S].astype(np.int32)
    p = torch.full((S + 2, *shape), 7.0, device="cuda")
    if states is not None:
        p[torch.from_numpy(rows).long().cuda()] = f32(states)
    return p, torch.from_numpy(rows).cuda()


def rest(p, rows):
    keep = torch.ones(p.shape[0], dtype=torch.bool)
    keep[rows.cpu().long()] = False
    return p.cpu()[keep]


# ---- rotary ------------------------------------------------------------------------------------
def turn(x, positions, frequencies, magnitude=1.0, interleaved=False, inverse=False):
    """x [T, heads, D] with its first pairs turned, in 64 bits."""
    n, out = len(frequencies), np.array(x, dtype=np.float64)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    angle = positions.astype(np.float64)[:, None, None] * frequencies * (-1.0 if inverse else 1.0)
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    p, q = out[..., a].copy(), out[..., b].copy()
    out[..., a], out[..., b] = p * c - q * s, q * c + p * s
    return out
