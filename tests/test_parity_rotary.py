"""GPU parity of rotary positions against the 64-bit reference. The bound: a cosine or sine is off by the rounding of
its angle (at most 2^-25 half turns, pi 2^-25) and of itself (2^-23), a result by that times the pair's magnitudes and
a few roundings: 2^-21 magnitude (|a| + |b|), and half a step of its type."""
import numpy as np
import pytest
import torch

import linear_cases as lc
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def expect(got, x, pos, f, magnitude, interleaved, inverse):
    want = lc.turn(x, pos, f, magnitude, interleaved, inverse)
    size, n = np.abs(x).astype(np.float64), len(f)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    pair = (size[..., a] + size[..., b]) * magnitude
    tol = np.zeros_like(size)
    tol[..., a], tol[..., b] = pair, pair
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= 2.0 ** -21 * tol + torch.finfo(got.dtype).eps / 2 * np.abs(want))
    assert np.array_equal(got.double().cpu().numpy()[..., 2 * n:], x[..., 2 * n:])


def run(T, H, HK, D, turned, dtype, *, interleaved=False, inverse=False, magnitude=1.0, layout="rows", in_place=False, far=5000, seed=0):
    r = np.random.default_rng(seed)
    q, k = lc.values(r.normal(size=(T, H, D)), dtype), lc.values(r.normal(size=(T, max(HK, 1), D)), dtype)
    pos = r.integers(-far // 10, far, size=T).astype(np.int32)
    f = gdn.rotary_frequencies(turned, 10000.0, scaling="linear", factor=1.7)
    tq, tk = lc.put(q, dtype, layout), lc.put(k, dtype, layout) if HK else None
    kw = {"interleaved": interleaved, "inverse": inverse, "magnitude": magnitude}
    if not in_place:
        kw["q_out"] = lc.put(np.full_like(q, np.nan), dtype, layout)
        kw["k_out"] = lc.put(np.full_like(k, np.nan), dtype, layout) if HK else None
    oq, ok = gdn.gdn_rotary(tq, tk, torch.from_numpy(pos).cuda(), f, **kw)
    torch.cuda.synchronize()
    fr = f.cpu().numpy()
    expect(oq, q, pos, fr, magnitude, interleaved, inverse)
    if HK:
        expect(ok, k, pos, fr, magnitude, interleaved, inverse)
    else:
        assert ok is None
    if not in_place:
        assert np.array_equal(tq.double().cpu().numpy(), q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,HK,D,turned", [(1, 1, 0, 2, 2), (7, 3, 1, 64, 64), (65, 32, 8, 128, 128), (33, 5, 5, 96, 24), (130, 2, 3, 80, 46),
                                             (19, 4, 2, 50, 50), (300, 12, 12, 128, 64), (2, 40, 16, 256, 96)])
def test_turns(T, H, HK, D, turned, interleaved, dtype):
    run(T, H, HK, D, turned, dtype, interleaved=interleaved, seed=T)


@pytest.mark.parametrize("layout", ["dense", "odd", "heads"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(layout, in_place, interleaved):
    run(40, 3, 2, 64, 32, "bf16", layout=layout, in_place=in_place, interleaved=interleaved)
    run(41, 3, 2, 72, 48, "f32", layout=layout, in_place=in_place, interleaved=interleaved)


@pytest.mark.parametrize("far", [1 << 20, 1 << 24])
def test_far_positions(far):
    """The reference's own angle is off by far 2^-53; an angle in fp32 would be off by far 2^-24."""
    run(50, 2, 1, 64, 64, "f32", far=far)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(interleaved):
    run(60, 3, 3, 64, 40, "f32", interleaved=interleaved, inverse=True, magnitude=1.4)
    x = torch.randn(20, 2, 64, device="cuda")
    pos, f = torch.arange(20, dtype=torch.int32, device="cuda"), gdn.rotary_frequencies(64)
    there, _ = gdn.gdn_rotary(x, None, pos, f, q_out=torch.empty_like(x), interleaved=interleaved)
    back, _ = gdn.gdn_rotary(there, None, pos, f, q_out=torch.empty_like(x), interleaved=interleaved, inverse=True)
    assert torch.allclose(back, x, atol=4e-6)


def test_frequencies_of_every_size():
    """Frequencies above a turn a position, negative, tiny and zero."""
    f = np.array([0.0, 1e-320, 1e-30, 3e-9, 0.5, -0.7, 3.0, 2 * np.pi, 7.5, -100.25, 12345.678, 1e9])
    x = np.random.default_rng(2).normal(size=(11, 1, 24))
    pos = np.arange(-5, 6).astype(np.int32)
    t = torch.from_numpy(x).float().cuda()
    out, _ = gdn.gdn_rotary(t, None, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), q_out=torch.empty_like(t))
    want = lc.turn(t.double().cpu().numpy(), pos, f)
    # the angle's rounding in the reference's own product: |pos f| 2^-53, five positions of 1e9 radians
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -21 * np.abs(x).max() * 2 + 5e9 * 2.0 ** -52 * 8)


def test_other_streams_and_graphs():
    x = torch.randn(100, 4, 64, device="cuda")
    out, pos, f = torch.empty_like(x), torch.arange(100, dtype=torch.int32, device="cuda"), gdn.rotary_frequencies(32)
    call = gdn.gdn_rotary(x, None, pos, f, q_out=out, prepare=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(s)
    s.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
