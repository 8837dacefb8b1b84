"""gdn_beam_select on logits of any finite size: rows of one large value, a few large values among ordinary ones, and
forbidden tokens marked by a large negative finite value instead of minus infinity. Within the bounds of
beam_reference, which do not depend on the logits' size: differences to the row's maximum are exact in 64 bits, and
a sum of equal exponentials is a count."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import test_parity_beam as beam

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def product_error(m):
    """What rounding to fp32 takes off m log2(e): the scale by which a sum of 2^(m log2(e) - rounded) is off."""
    f = np.float32(1.4426950408889634)
    with np.errstate(over="ignore"):
        return float(np.float32(m)) * float(f) - float(np.float32(m) * f)


# fp32 values whose product_error lies where 2^-error or a sum of 2^error leaves the normal fp32 numbers
LARGE_F32 = [2800010240.0, 2800012544.0, 2800028160.0, 2800061696.0, -2800010240.0, -2800012544.0, 2800001024.0, 2800001536.0]
LARGE_BF16 = [1509949440.0, 1619001344.0, 1702887424.0, 3405774848.0, -1509949440.0, 2348810240.0]
COMMON = [-1e4, -1e9, -1e30, 1e9, 1e30]


def test_the_large_values_are_what_they_are_for():
    e = [product_error(v) for v in LARGE_F32]
    assert any(-128 < v < -126 for v in e) and any(124 < v < 126 for v in e) and any(126 < v < 128 for v in e)


def _value(v, dtype):
    return float(torch.tensor(v).to(TYPES[dtype]).float())


def _cases():
    for v in LARGE_F32 + COMMON + [float(np.finfo(np.float32).min), float(np.finfo(np.float32).max)]:
        yield "f32", v
    for v in LARGE_BF16 + COMMON + [float(torch.finfo(torch.bfloat16).min), float(torch.finfo(torch.bfloat16).max)]:
        yield "bf16", v


@pytest.mark.parametrize("V", [300, 20003])
@pytest.mark.parametrize("dtype,value", list(_cases()))
def test_rows_of_one_value(dtype, value, V):
    x = torch.full((4, V), value, dtype=TYPES[dtype], device="cuda")
    got = beam._check(x, np.array([[0.0, -0.25, -0.5, -30.0]], dtype=np.float32), 8)
    assert list(got[1][0]) == [0] * 8 and list(got[2][0]) == list(range(8))
    assert abs(got[0][0, 0] + np.log(V)) <= ref.LSE_BOUND + 2.0 ** -24 * np.log(V)


def mixed_rows(R, V, dtype, value, share, seed):
    """Ordinary logits with `value` in a share of the places, as an array of the type's values."""
    r = np.random.default_rng(seed)
    x = 2.5 * r.normal(size=(R, V))
    x[r.random((R, V)) < share] = value
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])


MASKS = {"f32": [-1e4, -1e9, -2800010240.0, -1e30, float(np.finfo(np.float32).min)],
         "bf16": [-1e4, -1e9, -1509949440.0, -1e30, float(torch.finfo(torch.bfloat16).min)]}
MASK_CASES = [(t, v) for t in MASKS for v in MASKS[t]]


@pytest.mark.parametrize("share,K", [(0.5, 12), (0.9, 12), (0.9985, 12), (0.9985, 40), (1.0, 12)])
@pytest.mark.parametrize("dtype,mask", MASK_CASES)
def test_forbidden_by_a_finite_value(dtype, mask, share, K):
    """K of 40 asks for more candidates than the rows allow: masked tokens follow, at their distance."""
    x = mixed_rows(8, 6001, dtype, mask, share, 3)
    x[3] = _value(mask, dtype)                       # a row without any allowed token
    beam._check(x.cuda(), beam._scores(2, 4, 3), K)


@pytest.mark.parametrize("dtype,value", [(t, v) for t, vs in (("f32", LARGE_F32[:4]), ("bf16", LARGE_BF16[:4])) for v in vs])
def test_a_few_large_values(dtype, value):
    """They share their row's whole probability; the others follow at their distance."""
    x = mixed_rows(8, 6001, dtype, value, 0.0008, 4)
    x[:, 17] = _value(value, dtype)
    beam._check(x.cuda(), beam._scores(2, 4, 4), 4)
