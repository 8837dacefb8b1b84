"""The example model end to end: the scores that beam search accumulates over prompt scan, decode steps,
selections and state moves are those of one scan over prompt and continuation, and its training step learns.

The two ways compute the same sums in fp32 in another order: three layers of products over 64 to 128 terms and a
scan of at most 50 tokens, each off by about its terms' count in units of 2^-24 of magnitudes of order 10, below
1e-4 a logit and 2 x 8 x 1e-4 over eight tokens; PyTorch's fp32 matrix product stays in full fp32 by default."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams,seed", [(4, 0), (1, 1), (9, 2)])
def test_search_scores_are_the_sequences_own(beams, seed):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import mamba_beam_search as ex
    model = ex.Model(seed=seed)
    prompts = [[5, 17, 301], [9] * 40 + [2, 3], [44], [7, 8]]
    scores, history = ex.beam_search(model, prompts, beams, steps=8)
    again = ex.rescore(model, prompts, history)
    assert torch.all(torch.isfinite(scores))
    assert float((scores.cpu().double() - again).abs().max()) < 2e-3
    assert torch.all(scores[:, :-1] >= scores[:, 1:])
    for b in range(len(prompts)):
        assert len({tuple(h) for h in history[b].tolist()}) == beams


def test_greedy_is_one_beam_of_the_decode():
    import mamba_beam_search as ex
    model = ex.Model(seed=3)
    prompt = [3, 1, 4, 1, 5]
    _, history = ex.beam_search(model, [prompt], beams=1, steps=6, eos=0)
    tokens = list(prompt)
    for t in history[0, 0].tolist():
        if t < 0:
            break
        pools = [torch.zeros(1, l.D, l.N, device="cuda") for l in model.layers]
        logits, _ = model.run(torch.tensor(tokens, device="cuda"), [len(tokens)], pools, None)
        assert int(logits[-1].argmax()) == t
        tokens.append(t)


def test_training_learns():
    import mamba_beam_search as ex
    losses = ex.train()
    assert losses[-1] < 0.7 * losses[0]
