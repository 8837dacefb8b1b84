"""Log decays at their limit over segments of more than 29000 tokens: their sum passes what 64 bits hold in steps of 2^-40
(2^23 powers of two), and what lies before a segment has to stay forgotten."""
import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_segments_that_forget_everything(dtype):
    """g = -200: o_t = scale (q_t . k_t) v_t, whatever the tokens and the state before."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    T, HV, K, V = 65536, 304, 16, 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    q, k, v = n(T, 1, K), n(T, 1, K), n(T, HV, V)
    start = torch.randn(1, HV, V, K, generator=gen, device="cuda")
    o, final = torch.full_like(v, float("nan")), torch.full_like(start, float("nan"))
    ws = gdn.linear_attention_workspace(T, 1, HV, K, V, dtype=dtype)
    gdn.gdn_linear_attention(q, k, v, torch.full((HV,), -200.0, device="cuda"), o, initial_state=start, final_state=final, workspace=ws)
    torch.cuda.synchronize()
    assert ws is not None or dtype == torch.bfloat16                      # in fp32 the sequence is cut
    terms = (q.double() * k.double())[:, 0] * K ** -0.5
    want, size = terms.sum(-1)[:, None, None] * v.double(), terms.abs().sum(-1)[:, None, None] * v.double().abs()
    # K additions and a few roundings, with bf16 inputs two bf16 numbers of a score and of a state, and the output's rounding
    u = (K + 32) * 2.0 ** -23 + (2.0 ** -16 if dtype == torch.bfloat16 else 0.0)
    assert bool(((o.double() - want).abs() <= u * size + torch.finfo(dtype).eps / 2 * want.abs()).all())
    want = v[-1].double()[:, :, None] * k[-1].double()
    assert bool(((final[0].double() - want).abs() <= 2.0 ** -20 * want.abs()).all())
