"""Linear attention's accuracy against 64 bits in relative L2 norm, for heads that remember everything, a thousand tokens, twenty,
and two. The bounds of linear_cases grow with the sequence and take dg's terms up to its end, which hides most wrong dg
and a factor that is off by 1e-7 in every chunk; these do not.

The limits of states and outputs in fp32 are twice the largest figures measured beside the constants in linear_chunk.cu and
linear_common.cuh (states 1.9e-7 with bf16 inputs, 2.6e-7 in fp32; outputs 2.5e-6 and 2.3e-7). bf16 outputs and gradients may be 3%
further off than the exact ones rounded. `bias` is the mean of the relative error weighted by the values' squares: 1.3e-7 at
most. What dg may be off by follows from these and from the rounding of its scores (dg_limit): the shorter the sequence or the
memory, the more of its sums cancels."""
import numpy as np
import pytest
import torch

import linear_cases as lc

CHUNK = 128
MEMORIES = [(0.0, 0.0), (1e-4, 1e-3), (0.05, 0.05), (0.5, 0.5)]
STATES = {"bf16": 2 * 1.9e-7, "f32": 2 * 2.6e-7}
OUTPUTS = {"bf16": 2 * 2.5e-6, "f32": 2 * 2.3e-7}
BIAS = 2 * 1.3e-7


def off(got, ref):
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


def bias(got, ref):
    return float(((got - ref) * ref).sum() / (ref * ref).sum())


def case(lengths, H, HV, K, V, dtype, memory, seed=3):
    c = lc.make(lengths, H, HV, K, V, dtype, seed, decay=(max(memory[0], 1e-9), max(memory[1], 1e-9)))
    if memory[1] == 0.0:
        c["g"][:] = 0.0
    elif memory[0] == memory[1]:
        c["g"] = (c["g"] * np.random.default_rng(4).uniform(1.0, 1.2, size=c["g"].shape)).astype(np.float32).astype(np.float64)
    return c


def borders(c):
    """<D, S> at the end of every chunk of every sequence [tokens of the chunk's end, HV], D with the decay of the token behind."""
    q, k, v, do, sc = c["q"], c["k"], c["v"], c["do"], c["scale"]
    T, HV, V = v.shape
    G = HV // q.shape[1]
    a, wide, out, at = np.exp(c["g"]), lambda x: np.repeat(x, G, 0), np.zeros((T, HV)), 0
    for s, n in enumerate(c["lengths"]):
        S, D, keep = c["initial"][s].copy(), c["d_final"][s].copy(), {}
        for t in range(at, at + n):
            S = a[t][:, None, None] * S + v[t][:, :, None] * wide(k[t])[:, None, :]
            if (t - at) % CHUNK == CHUNK - 1 or t == at + n - 1:
                keep[t] = S
        for t in range(at + n - 1, at - 1, -1):
            if t in keep:
                out[t] = (D * keep[t]).sum((1, 2))
            D = a[t][:, None, None] * (D + sc * do[t][:, :, None] * wide(q[t])[:, None, :])
        at += n
    return out


def by_chunks(c, ref, edge, sign=-1.0):
    """dg as a sum to the end of each chunk and the product there."""
    T, HV, _ = c["v"].shape
    wide = lambda x: np.repeat(x, HV // c["q"].shape[1], 1)
    terms = (wide(c["q"]) * ref["dq_heads"]).sum(-1) + sign * (wide(c["k"]) * ref["dk_heads"]).sum(-1)
    dg, at = np.zeros((T, HV)), 0
    for n in c["lengths"]:
        for first in range(at, at + n, CHUNK):
            last = min(first + CHUNK, at + n)
            dg[first:last] = terms[first:last][::-1].cumsum(0)[::-1] + edge[last - 1]
        at += n
    return dg


def magnitudes(c):
    """The sum of the magnitudes of what the kernels for bf16 add up for dg: a row's terms to the end of its chunk, and the
    product there."""
    m = {k: np.abs(x) if isinstance(x, np.ndarray) and k != "g" else x for k, x in c.items()}
    return by_chunks(m, lc.backward(m), borders(m), sign=1.0)


def dg_limit(c, ref, edge):
    """The relative norm of dg's error. dg_t adds up q.dq - k.dk over the rows behind it in its chunk, and the border's product.
    With M_rs = (scale do_r.v_s e^{G_r - G_s}) (q_r.k_s), both q_r.dq_r and k_s.dk_s have the sum of their M in
    them. With bf16 inputs each score times decay is two bf16 numbers: a rounding is uniform over a step, 2^-8 / sqrt(3) of its power of
    two in the mean square, and the second one's error that of the first one's remainder: 2^-16 / 3 of M, independent for each r and s
    and of the two sums. Beside that dq and dk are off by what OUTPUTS (fp32) and STATES allow in fp32, in any direction
    against q and k (the square root of K of it along them) or in proportion; the border's two states by STATES."""
    q, k, v, do, K = c["q"], c["k"], c["v"], c["do"], c["q"].shape[2]
    T, HV, _ = v.shape
    G, eps = HV // q.shape[1], 2.0 ** -16 / 3 if c["dtype"] == "bf16" else 0.0
    u = STATES[c["dtype"]] + OUTPUTS["f32"]
    square, at = np.zeros((T, HV)), 0
    for n in c["lengths"]:
        for first in range(at, at + n, CHUNK):
            rows = slice(first, min(first + CHUNK, at + n))
            for h in range(HV):
                qh, kh, g = q[rows, h // G], k[rows, h // G], np.cumsum(c["g"][rows, h])
                M = c["scale"] * (do[rows, h] @ v[rows, h].T) * (qh @ kh.T) * np.exp(np.minimum(g[:, None] - g[None, :], 0.0))
                M = np.tril(M) ** 2 * eps ** 2
                own = M.sum(1) + M.sum(0)
                for x, y in ((qh, ref["dq_heads"][rows, h]), (kh, ref["dk_heads"][rows, h])):
                    own += u ** 2 * ((x * x).sum(-1) * (y * y).sum(-1) / K + (x * y).sum(-1) ** 2)
                square[rows, h] = own[::-1].cumsum()[::-1] + (2 * STATES[c["dtype"]] * edge[rows.stop - 1, h]) ** 2
        at += n
    return float(np.sqrt(square.sum()) / np.linalg.norm(ref["dg"]))


@pytest.mark.parametrize("memory", MEMORIES[1:])
@pytest.mark.parametrize("lengths", [[700], [500, 300]])
def test_a_wrong_border_is_far_outside_the_limits(lengths, memory):
    """The product at the chunks' ends left out, at the inner ends only, without its decay, or all zeros: none would pass."""
    c = case(lengths, 1, 2, 32, 32, "bf16", memory)
    ref, edge = lc.backward(c), borders(c)
    assert off(by_chunks(c, ref, edge), ref["dg"]) < 1e-11
    ends, inner = np.cumsum(lengths) - 1, edge.copy()
    inner[[t for t in range(len(edge)) if t not in ends]] = 0.0
    late = edge.copy()
    late[:-1] /= np.exp(c["g"][1:])                          # each inner product before the next token's decay
    late[ends] = edge[ends]
    limit = dg_limit(c, ref, edge)
    tol, u = magnitudes(c), (CHUNK + 32 + 32 + 32) * 2.0 ** -23 + 2.0 ** -16
    wrong = {"none": np.zeros_like(edge), "inner": inner, "zeros": None} | ({"decay": late} if memory[0] > 1e-3 else {})
    for name, e in wrong.items():
        got = np.zeros_like(ref["dg"]) if e is None else by_chunks(c, ref, e)
        assert off(got, ref["dg"]) > 1000 * limit, name
        assert np.any(np.abs(got - ref["dg"]) > u * tol), name


def _numpy(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("memory", MEMORIES)
@pytest.mark.parametrize("lengths,H,HV,K,V", [([1100, 900], 1, 2, 64, 128), ([2048], 1, 1, 128, 64), ([160] * 6, 1, 2, 64, 64)])
def test_errors_in_norm(lengths, H, HV, K, V, memory, dtype):
    from test_parity_linear import run_backward, run_forward
    c = case(lengths, H, HV, K, V, dtype, memory)
    ref = lc.forward(c) | lc.backward(c)
    got = {n: _numpy(t) for n, t in (run_forward(c) | run_backward(c)).items()}
    if dtype == "bf16":
        o32 = _numpy(run_forward(c, out="f32")["o"])
        assert off(o32, ref["o"]) < OUTPUTS[dtype]
    for n in ("final", "d_initial"):
        assert off(got[n], ref[n]) < STATES[dtype], (n, off(got[n], ref[n]))
        assert abs(bias(got[n], ref[n])) < BIAS, (n, bias(got[n], ref[n]))
    for n in ("o", "dq", "dk", "dv"):
        limit = OUTPUTS[dtype]
        if dtype == "bf16":
            limit = 1.03 * off(lc.values(ref[n], dtype), ref[n])
        assert off(got[n], ref[n]) < limit, (n, off(got[n], ref[n]), limit)
    limit = dg_limit(c, ref, borders(c))
    assert off(got["dg"], ref["dg"]) < limit, (off(got["dg"], ref["dg"]), limit)


@pytest.mark.gpu
@pytest.mark.parametrize("memory", MEMORIES)
@pytest.mark.parametrize("lengths,H,HV,K,V", [([1100, 900], 1, 2, 64, 128), ([160] * 6, 1, 2, 64, 64)])
def test_dg_within_what_a_chunk_adds_up(lengths, H, HV, K, V, memory):
    """Each dg of the kernel for bf16 inputs within the bound of linear_cases for sums that end with the chunk."""
    from test_parity_linear import run_backward
    c = case(lengths, H, HV, K, V, "bf16", memory)
    got, ref = _numpy(run_backward(c)["dg"]), lc.backward(c)["dg"]
    u = (CHUNK + K + V + 32) * 2.0 ** -23 + 2.0 ** -16
    # (its terms' own states have been through all tokens: their error is part of them)
    u += max(lengths) * 2.0 ** -23
    assert np.all(np.abs(got - ref) <= u * magnitudes(c) + 2.0 ** -24 * np.abs(ref))
