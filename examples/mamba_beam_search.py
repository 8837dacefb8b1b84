"""A small Mamba-1 language model with random weights: prompts, beam search and a training step.

Runs the library's sequence and search operators together, as a serving or training program would:

  prompts   mamba_selective_scan over packed prompts of different lengths; every layer's final states go
            to the state pool's rows of the requests' first beams
  search    per token: mamba_selective_scan_decode over the pool (its rows are the slots), gdn_beam_select
            over the logits in slot order, gdn_beam_reorder of all layers' pools
  training  mamba_selective_scan and mamba_selective_scan_backward inside a gradient step

  python examples/mamba_beam_search.py            (a GB300; prints the best continuations and a falling loss)
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ssm_recurrent_decode_gb300 as gdn  # noqa: E402


class Layer:
    """x, z = W_in u; dt = softplus(W_dt u + b); B, C = W_bc u; y = scan(x, dt, B, C) gated by z; u + W_out y."""

    def __init__(self, width, D, N, g):
        r = lambda *s, scale=1.0: scale * torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[-1])
        self.D, self.N = D, N
        self.W_in, self.W_dt, self.W_bc, self.W_out = r(2 * D, width), r(D, width), r(2 * N, width), r(width, D)
        self.dt_bias = torch.log(torch.expm1(torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))))
        self.A = -torch.arange(1, N + 1, dtype=torch.float32, device="cuda").repeat(D, 1).contiguous()
        self.Dskip = torch.ones(D, device="cuda")

    def inputs(self, u):
        """Row views x, z of one projection, and dt, B, C."""
        u = u / (u.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        xz, bc = u @ self.W_in.T, u @ self.W_bc.T
        dt = torch.nn.functional.softplus(u @ self.W_dt.T + self.dt_bias)
        return xz[:, :self.D], xz[:, self.D:], dt, bc[:, :self.N], bc[:, self.N:]

    def scan(self, u, cu_seqlens, h_last, state_indices):
        x, z, dt, B, C = self.inputs(u)
        y = torch.empty(u.shape[0], self.D, device="cuda")
        ws = gdn.mamba_scan_workspace(u.shape[0], self.D, self.N, sequences=cu_seqlens.numel() - 1, uniform=False)
        gdn.mamba_selective_scan(x, dt, self.A, B, C, y, Dskip=self.Dskip, z=z, cu_seqlens=cu_seqlens, h_last=h_last,
                                 state_indices=state_indices, workspace=ws)
        return u + y @ self.W_out.T

    def step(self, u, h):
        x, z, dt, B, C = (t.contiguous() for t in self.inputs(u))
        y = torch.empty_like(x)
        gdn.mamba_selective_scan_decode(x, dt, self.A, B, C, h, y, Dskip=self.Dskip, z=z)
        return u + y @ self.W_out.T


class Model:
    def __init__(self, vocab=1000, width=64, D=128, N=16, layers=3, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.width = vocab, width
        self.embed = torch.randn(vocab, width, generator=g, device="cuda")
        self.head = 2.0 * torch.randn(vocab, width, generator=g, device="cuda") / math.sqrt(width)
        self.layers = [Layer(width, D, N, g) for _ in range(layers)]

    def logits(self, u):
        return (u / (u.square().mean(-1, keepdim=True) + 1e-5).sqrt()) @ self.head.T

    def run(self, tokens, lengths, pools, rows):
        """Logits of every token of packed sequences; each layer's final states go to its pool's rows."""
        cu = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        u = self.embed[tokens]
        for layer, pool in zip(self.layers, pools):
            u = layer.scan(u, cu, pool, rows)
        return self.logits(u), cu

    def step(self, tokens, pools):
        u = self.embed[tokens]
        for layer, pool in zip(self.layers, pools):
            u = layer.step(u, pool)
        return self.logits(u)


def beam_search(model, prompts, beams=4, steps=8, eos=1):
    """The `beams` best continuations of each prompt (a list of token lists): scores [batch, beams], tokens
    [batch, beams, steps] (-1 behind a continuation's end)."""
    batch = len(prompts)
    slots_n = batch * beams
    pools = [torch.zeros(slots_n, l.D, l.N, device="cuda") for l in model.layers]
    slots = torch.arange(slots_n, dtype=torch.int32, device="cuda").view(batch, beams)
    other = torch.empty_like(slots)
    tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
    logits, cu = model.run(tokens, [len(p) for p in prompts], pools, slots[:, 0].contiguous())

    # the first selection: one beam per request holds a state, the others are dead
    scores = torch.full((batch, beams), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    rows = torch.arange(batch, dtype=torch.int32, device="cuda").view(batch, 1).repeat(1, beams)
    logits = logits[cu[1:].long() - 1].contiguous()
    finished = torch.zeros(batch, beams, dtype=torch.uint8, device="cuda")
    history = torch.full((batch, beams, steps), -1, dtype=torch.int32, device="cuda")
    ws = gdn.beam_select_workspace(batch, beams, model.vocab, beams)
    for step in range(steps):
        new_scores, new_finished = torch.empty_like(scores), torch.empty_like(finished)
        parents, chosen = torch.empty_like(slots), torch.empty_like(slots)
        gdn.gdn_beam_select(logits, scores, new_scores, parents, chosen, rows=rows, finished=finished, eos_token=eos,
                            out_finished=new_finished, workspace=ws)
        gdn.gdn_beam_reorder(pools, slots, parents, other)
        slots, other = other, slots
        # what each new beam has said so far, its new token behind (nothing behind an end)
        gone = torch.gather(finished, 1, parents.clamp_min(0).long()).bool()
        history = torch.gather(history, 1, parents.clamp_min(0).long()[:, :, None].expand(-1, -1, steps)).contiguous()
        history[:, :, step] = torch.where(gone, -1, chosen)
        scores, finished = new_scores, new_finished
        if step + 1 < steps:
            # the decode's rows are the pool's slots: a beam's token goes to its slot's row, its logits come from there
            by_slot = torch.zeros(slots_n, dtype=torch.int64, device="cuda")
            by_slot[slots.view(-1).long()] = chosen.view(-1).clamp_min(0).long()
            logits = model.step(by_slot, pools)
            rows = slots
    return scores, history


def rescore(model, prompts, history):
    """The same continuations' scores from one packed scan over prompt and continuation."""
    batch, beams, _ = history.shape
    seqs, starts = [], []
    for b in range(batch):
        for j in range(beams):
            said = [t for t in history[b, j].tolist() if t >= 0]
            seqs.append(list(prompts[b]) + said)
            starts.append(len(prompts[b]))
    pools = [torch.zeros(len(seqs), l.D, l.N, device="cuda") for l in model.layers]
    logits, cu = model.run(torch.tensor([t for s in seqs for t in s], device="cuda"), [len(s) for s in seqs], pools, None)
    logp = torch.log_softmax(logits.double(), -1)
    out = []
    for i, (s, start) in enumerate(zip(seqs, starts)):
        at = int(cu[i])
        out.append(sum(float(logp[at + t - 1, s[t]]) for t in range(start, len(s))))
    return torch.tensor(out).view(batch, beams)


def train(steps=20, sequences=4, length=96, D=64, N=16, lr=0.05, seed=0):
    """Fits A, the skip weights and the step sizes of one scan to another's outputs; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sequences * length
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, z, B, C = n(T, D), n(T, D), n(T, N), n(T, N)
    def make():
        return -torch.exp(0.5 * n(D, N)), 1.0 + 0.3 * n(D), 0.02 + 0.05 * torch.rand(D, generator=g, device="cuda")
    def forward(A, skip, step, y):
        dt = step.expand(T, D).contiguous()
        gdn.mamba_selective_scan(x, dt, A, B, C, y, Dskip=skip, z=z, sequences=sequences,
                                 workspace=gdn.mamba_scan_workspace(T, D, N, sequences=sequences))
        return dt
    target, y = torch.empty(T, D, device="cuda"), torch.empty(T, D, device="cuda")
    forward(*make(), target)
    A, skip, step = make()
    dA, dskip, ddt = torch.empty_like(A), torch.empty_like(skip), torch.empty(T, D, device="cuda")
    ws = gdn.mamba_scan_workspace(T, D, N, sequences=sequences, backward=True)
    losses = []
    for _ in range(steps):
        dt = forward(A, skip, step, y)
        off = y - target
        losses.append(float(off.square().mean()))
        gdn.mamba_selective_scan_backward(x, dt, A, B, C, off * (2.0 / off.numel()), Dskip=skip, z=z, sequences=sequences,
                                          dA=dA, dDskip=dskip, ddt=ddt, workspace=ws)
        A = A - lr * D * dA
        skip = skip - lr * D * dskip
        step = (step - 0.01 * lr * D * ddt.sum(0)).clamp_min(1e-3)
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--beams", type=int, default=4)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    model = Model()
    prompts = [[5, 17, 301], [9] * 40 + [2, 3], [44]]
    scores, history = beam_search(model, prompts, a.beams, a.steps)
    again = rescore(model, prompts, history)
    for b, prompt in enumerate(prompts):
        print(f"prompt of {len(prompt)} tokens")
        for j in range(a.beams):
            print(f"  {float(scores[b, j]):9.4f} (one scan: {float(again[b, j]):9.4f})  {history[b, j].tolist()}")
    losses = train()
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
