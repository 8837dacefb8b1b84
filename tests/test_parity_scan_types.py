"""The gradients in both types over state sizes that take every instance of the kernels (2, 4, 8, 16 and 32 lanes along
the state), in one chunk and across several, and guard bands and the index-checking build for those instances that
test_canaries_sequences does not run."""
import pytest
import torch

import test_canaries_sequences as canaries
import test_parity_scan as scan

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("N", [1, 3, 8, 13, 24, 32, 50, 64, 100, 128])
def test_bf16_gradients_over_state_sizes(N):
    scan._backward([5, 0, 70, 1], 37, N, "bf16", seed=N)


@pytest.mark.parametrize("N", [3, 8, 16, 24, 50, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_across_chunks(N, dtype):
    """Several chunks, sequences across their borders, channels that do not fill a tile."""
    scan._backward([5, 0, 270, 1, 64], 37, N, dtype, seed=100 + N)


@pytest.mark.parametrize("N", [8, 24, 128])
@pytest.mark.parametrize("gate,skip,states", [(False, False, False), (True, False, True)])
def test_bf16_gradients_with_optional_inputs(N, gate, skip, states):
    scan._backward([40, 159], 130, N, "bf16", gate=gate, skip=skip, states=states, seed=N)


@pytest.mark.parametrize("N", [7, 31, 127])
def test_bf16_gradients_of_strided_rows(N):
    scan._backward([50, 90], 61, N, "bf16", strided=True, seed=N)


CASES = [([40, 41, 200], 130, 4, "bf16"), ([90, 0, 77], 70, 8, "bf16"), ([64, 1, 130], 72, 24, "bf16"), ([64, 1, 130], 72, 32, "f32"),
         ([300], 48, 64, "f32")]


@pytest.mark.parametrize("lengths,D,N,dtype", CASES)
def test_guard_bands_forward(lengths, D, N, dtype):
    canaries.test_scan(lengths, D, N, dtype)


@pytest.mark.parametrize("lengths,D,N,dtype", CASES)
def test_guard_bands_backward(lengths, D, N, dtype):
    canaries.test_scan_backward(lengths, D, N, dtype)


def test_gradients_on_another_stream_and_in_a_graph():
    lengths, D, N = [70, 0, 90], 64, 24
    c = scan.sc.make(lengths, D, N, "bf16", 14)
    d = scan._dev(c, "bf16")
    h0, dhl = torch.from_numpy(c["h0"]).cuda(), torch.from_numpy(c["dh_last"]).cuda()
    ws, cu = scan._workspace(lengths, D, N, False, True), scan._cu(lengths)
    bf = lambda w: torch.zeros(160, w, dtype=torch.bfloat16, device="cuda")
    new = lambda: {"dx": bf(D), "ddt": bf(D), "dz": bf(D), "dBm": bf(N), "dCm": bf(N), "dA": torch.zeros(D, N, device="cuda"),
                   "dDskip": torch.zeros(D, device="cuda"), "dh0": torch.zeros_like(h0)}

    def call(g, stream=None):
        scan.gdn.mamba_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], Dskip=d["Dskip"], z=d["z"],
                                               cu_seqlens=cu, h0=h0, dh_last=dhl, workspace=ws, stream=stream, **g)
    plain, other, captured = new(), new(), new()
    call(plain)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(other, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(captured)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in plain:
        assert torch.equal(other[k], plain[k]) and torch.equal(captured[k], plain[k]), k
