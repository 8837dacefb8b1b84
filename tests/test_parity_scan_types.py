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
