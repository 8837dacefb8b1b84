"""What the binding of linear attention refuses before it asks for a GPU."""
import pytest
import torch

import ssm_recurrent_decode_gb300 as gdn


def test_a_step_refuses_a_magnitude_of_zero():
    """In the C struct 0 selects 1; given as a number it would turn q and k into what was not asked for (gdn_rotary
    refuses it too)."""
    t = torch.zeros(4, 2, 16)
    with pytest.raises(ValueError, match="magnitude"):
        gdn.gdn_linear_attention_step(t, t, t, torch.zeros(2), torch.zeros(4, 2, 16, 16), t, positions=torch.zeros(4, dtype=torch.int32),
                                      frequencies=torch.ones(8, dtype=torch.float64), magnitude=0.0)


@pytest.mark.gpu
def test_bf16_outputs_of_fp32_inputs():
    import linear_cases as lc
    from test_parity_linear import compare, run_forward
    c = lc.make([140, 75], 2, 2, 64, 40, "f32", 19)
    compare(c, run_forward(c, out="bf16"))
