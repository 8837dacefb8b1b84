"""Inputs, references and error bounds of the selective-scan tests.

The bounds are derived from the arithmetic, not from results. Every output is a sum of products of
inputs and decays; with each factor replaced by its magnitude the 64-bit reference gives the sum of
the terms' magnitudes, `mag`. A term's relative error is at most that of its products: one decay per
token passed (the exponential's 2^-22 and its argument's rounding, |dt A| 2^-23, where the largest
|dt A| met counts) and a few roundings of 2^-24, so an output after L tokens is off by at most
(L + 8) (2 + max|dt A|) 2^-22 mag; sums over D channels or T tokens in fp32 add at most 2^-24 mag per
term added one after another. An output of a narrower type adds half a step of it."""
import numpy as np
import torch

import oracle

UNIT = 2.0 ** -22


def bf16_values(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def make(lengths, D, N, dtype, seed, *, gate=True, skip=True, states=True):
    """fp32 arrays holding values of `dtype` (the states and parameters stay fp32)."""
    r = np.random.default_rng(seed)
    T, S = sum(lengths), len(lengths)
    q = bf16_values if dtype == "bf16" else (lambda a: np.asarray(a, dtype=np.float32))
    c = {"x": q(r.normal(size=(T, D))), "dt": q(np.exp(r.uniform(np.log(1e-3), np.log(0.3), size=(T, D)))),
         "Bm": q(r.normal(size=(T, N))), "Cm": q(r.normal(size=(T, N))), "dy": q(r.normal(size=(T, D))),
         "A": (-np.exp(r.uniform(np.log(0.3), np.log(16.0), size=(D, N)))).astype(np.float32),
         "z": q(r.normal(size=(T, D))) if gate else None,
         "Dskip": r.normal(size=D).astype(np.float32) if skip else None,
         "h0": r.normal(size=(S, D, N)).astype(np.float32) if states else None,
         "dh_last": r.normal(size=(S, D, N)).astype(np.float32) if states else None}
    c["lengths"] = list(lengths)
    return c


def unit(c):
    """The relative error a term of this case may have: see the module text."""
    most = max(c["lengths"], default=0)
    worst = float(np.max(np.abs(c["dt"])) * np.max(np.abs(c["A"]))) if c["dt"].size else 0.0
    return (most + 8) * (2 + worst) * UNIT


def forward(c):
    """Reference outputs and the magnitudes of their sums."""
    kw = {"lengths": c["lengths"], "Dskip": c["Dskip"], "z": c["z"], "h0": c["h0"]}
    y, h = oracle.mamba_scan(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], **kw)
    ab = lambda v: None if v is None else np.abs(v)
    ym, hm = oracle.mamba_scan(ab(c["x"]), c["dt"], c["A"], ab(c["Bm"]), ab(c["Cm"]), lengths=c["lengths"],
                               Dskip=ab(c["Dskip"]), h0=ab(c["h0"]))
    if c["z"] is not None:
        z = c["z"].astype(np.float64)
        ym = ym * np.abs(z * oracle.sigmoid(z))
    return {"y": y, "h_last": h}, {"y": ym, "h_last": hm}


def backward(c):
    ab = lambda v: None if v is None else np.abs(v)
    args = (c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"])
    ref = oracle.mamba_scan_backward(*args, lengths=c["lengths"], Dskip=c["Dskip"], z=c["z"], h0=c["h0"],
                                     dh_last=c["dh_last"])
    dy = np.abs(c["dy"].astype(np.float64))
    if c["z"] is not None:
        z = c["z"].astype(np.float64)
        dy = dy * np.abs(z * oracle.sigmoid(z))
    # magnitudes: A enters the decays with its sign, the sums with its magnitude
    mag = oracle.mamba_scan_backward(ab(c["x"]), c["dt"], c["A"], ab(c["Bm"]), ab(c["Cm"]), dy, lengths=c["lengths"],
                                     Dskip=ab(c["Dskip"]), h0=ab(c["h0"]), dh_last=ab(c["dh_last"]))
    neg = oracle_ddt_magnitude(c, dy)
    mag["ddt"] = neg
    if c["z"] is not None:
        pre, _ = oracle.mamba_scan(ab(c["x"]), c["dt"], c["A"], ab(c["Bm"]), ab(c["Cm"]), lengths=c["lengths"],
                                   Dskip=ab(c["Dskip"]), h0=ab(c["h0"]))
        s = oracle.sigmoid(z)
        mag["dz"] = np.abs(c["dy"]) * pre * s * (1 + np.abs(z) * (1 - s))
    return ref, mag


def oracle_ddt_magnitude(c, dy):
    """sum of |x| |du| and |A| |w|: ddt of the magnitudes with A negative is their difference, so the second part
    is taken twice (ddt = x du + sum A w with A < 0, hence x du + sum |A| w = 2 x du - ddt)."""
    ab = lambda v: None if v is None else np.abs(v)
    m = oracle.mamba_scan_backward(ab(c["x"]), c["dt"], c["A"], ab(c["Bm"]), ab(c["Cm"]), dy, lengths=c["lengths"],
                                   Dskip=None, h0=ab(c["h0"]), dh_last=ab(c["dh_last"]))
    du = m["dx"] / np.maximum(c["dt"].astype(np.float64), 1e-30)
    return 2 * np.abs(c["x"]) * du - m["ddt"]


def check(name, got, ref, mag, u, dtype=torch.float32, terms=0):
    """|got - ref| within u mag, `terms` one-by-one fp32 additions, and half a step of the output's type."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    half = torch.finfo(dtype).eps / 2
    tol = (u + terms * 2.0 ** -24) * mag * (1 + half) + half * np.abs(ref) + 1e-37
    off = np.abs(got - ref)
    assert np.all(np.isfinite(got)), name
    assert np.all(off <= tol), (name, float(np.max(off / tol)), np.unravel_index(np.argmax(off / tol), off.shape))
