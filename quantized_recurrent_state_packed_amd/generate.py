"""Beam search with a small random linear-attention model, from ragged prompts to
sequences: every state-related step runs in the library.

    prompts --stepq_linear_prefill--> states --stepq_pack--> one slot a request
    last logits --stepq_beam_select--> tokens, parents --stepq_beam_reorder--> a slot a beam
    tokens --stepq_decode_step on the packed slots--> logits --select, reorder--> ...

    python -m quantized_recurrent_state_packed_amd.generate --bits 6 --beams 4 --steps 16

The model (embedding, per layer q, k, v, beta, gate and output projections,
logits) has random weights and stands in for whatever computes q, k, v from tokens.
"""
from __future__ import annotations

import argparse

import numpy as np

from . import beam
from . import stepq as S
from .linear import LinearAttention


class RandomModel:
    """Weights of a linear-attention language model, and what it computes around the states."""

    def __init__(self, vocab: int, width: int, layers: int, heads: int, d: int, seed: int = 0, device="cuda"):
        import torch
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(device)

        self.vocab, self.layers, self.H, self.D = vocab, layers, heads, d
        self.embedding = weight(vocab, width, scale=1.0)
        self.qkv = [weight(width, 3 * heads * d, scale=width ** -0.5) for _ in range(layers)]
        self.rates = [weight(width, 2 * heads, scale=width ** -0.5) for _ in range(layers)]
        self.out = [weight(heads * d, width, scale=2.0 * (heads * d) ** -0.5) for _ in range(layers)]
        self.head = weight(width, vocab, scale=2.0 * width ** -0.5)

    def inputs(self, layer: int, x):
        """x [T, width] -> q, k (unit norm), v [T, H, D], beta and gate [T, H]."""
        import torch
        q, k, v = (x @ self.qkv[layer]).unflatten(-1, (3, self.H, self.D)).unbind(1)
        q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
        beta, gate = torch.sigmoid(x @ self.rates[layer]).unflatten(-1, (2, self.H)).unbind(1)
        return q.contiguous(), k.contiguous(), v.contiguous(), beta.contiguous(), (0.5 + 0.5 * gate).contiguous()

    def logits(self, x):
        return x @ self.head

    def add(self, layer: int, x, o):
        """The residual stream after a layer, at unit size."""
        y = x + o.flatten(1) @ self.out[layer]
        return y / y.square().mean(-1, keepdim=True).sqrt()


class BeamGenerator:
    """Beam search over a batch of prompts; the states live in one packed pool per layer."""

    def __init__(self, model: RandomModel, batch: int, beams: int, layout: S.Layout, eos_token: int = 0, device="cuda"):
        import torch
        self.model, self.batch, self.beams, self.layout, self.eos = model, batch, beams, layout, eos_token
        self.attention = LinearAttention(model.H, model.D, rule="delta", dtype=torch.float32)
        self.select = beam.BeamSelect(batch, beams, model.vocab, beams, torch.float32, eos_token=eos_token, device=device)
        self.slots = torch.arange(batch * beams, dtype=torch.int32, device=device)
        self.next_slots = torch.empty_like(self.slots)
        self.pools = [layout.alloc(batch * beams, device=device) for _ in range(model.layers)]
        self.device = device

    def _check_prompts(self, prompts) -> None:
        def refuse(detail):
            raise S.StepqError(S.STEPQ_ERR_INVALID_ARG, "BeamGenerator", detail)

        if len(prompts) != self.batch:
            refuse(f"{len(prompts)} prompts for a batch of {self.batch}")
        for b, p in enumerate(prompts):
            if len(p) == 0:       # the first choice is made from the last token's logits
                refuse(f"request {b}'s prompt is empty")
            if min(p) < 0 or max(p) >= self.model.vocab:
                refuse(f"request {b}'s prompt has tokens outside of the vocabulary of {self.model.vocab}")

    def prefill(self, prompts):
        """Prompts (non-empty lists of tokens, one a request) into the first slot of every
        request; the last tokens' logits [batch, vocab]."""
        import torch
        self._check_prompts(prompts)
        lengths = [len(p) for p in prompts]
        cu = torch.tensor(np.r_[0, np.cumsum(lengths)], dtype=torch.int32, device=self.device)
        tokens = torch.tensor([t for p in prompts for t in p], device=self.device)
        first = self.slots.view(self.batch, self.beams)[:, 0].contiguous()
        order = torch.arange(self.batch, dtype=torch.int32, device=self.device)
        x = self.model.embedding[tokens]
        workspace = self.attention.workspace(self.batch, len(tokens), device=self.device)
        for layer, (pool, scales) in enumerate(self.pools):
            q, k, v, beta, gate = self.model.inputs(layer, x)
            states = self.attention.states(self.batch, device=self.device)
            o = torch.empty_like(v)
            self.attention.prefill(cu, q, k, v, beta, gate, order, states, o, workspace=workspace)
            S.stepq_pack(self.layout.handle, self.batch, first, self.batch * self.beams, states, pool, scales)
            x = self.model.add(layer, x, o)
        return self.model.logits(x[(cu[1:] - 1).long()])

    def step(self, tokens):
        """One token of every beam [batch * beams] through the packed states; its logits."""
        import torch
        x = self.model.embedding[tokens.long()]
        n = self.batch * self.beams
        for layer, (pool, scales) in enumerate(self.pools):
            q, k, v, beta, gate = self.model.inputs(layer, x)
            o = torch.empty_like(v)
            S.stepq_decode_step(self.layout.handle, n, self.slots, n, q, k, v, beta, gate, pool, scales, o)
            x = self.model.add(layer, x, o)
        return self.model.logits(x)

    def choose(self, logits, scores, finished):
        """The next tokens and parents, and every layer's slots brought in line with them."""
        tokens, parents, scores = self.select(logits, scores, finished=finished)
        buffers = [t for pair in self.pools for t in pair]
        beam.reorder(self.beams, self.slots, parents.view(-1), buffers, self.next_slots, num_slots=self.batch * self.beams)
        self.slots, self.next_slots = self.next_slots, self.slots
        return tokens.clone(), parents.long().clamp(min=0), scores.clone()

    def run(self, prompts, steps: int):
        """Sequences [batch, beams, steps] and scores [batch, beams], best first."""
        import torch
        b, k = self.batch, self.beams
        scores = torch.full((b, k), -float("inf"), device=self.device)
        scores[:, 0] = 0.0                       # the prompt's one state; the first choice forks it
        logits = self.prefill(prompts).repeat_interleave(k, 0)
        sequences = torch.empty(b, k, 0, dtype=torch.int32, device=self.device)
        finished = None
        for t in range(steps):
            tokens, parents, scores = self.choose(logits.contiguous(), scores.reshape(-1), finished)
            sequences = torch.cat([sequences.gather(1, parents[..., None].expand(b, k, t)), tokens[..., None]], -1)
            ended = tokens == self.eos
            if finished is not None:
                ended |= finished.view(b, k).gather(1, parents).bool()
            finished = ended.view(-1).to(torch.uint8)
            if t + 1 < steps:
                logits = self.step(tokens.clamp(min=0).view(-1))
        return sequences, scores


def main() -> None:
    import torch
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--bits", type=int, default=6, choices=(4, 6, 8, 16, 32))
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--beams", type=int, default=4)
    a.add_argument("--steps", type=int, default=16)
    a.add_argument("--heads", type=int, default=8)
    a.add_argument("--dim", type=int, default=64, choices=(16, 32, 64, 128))
    a.add_argument("--vocab", type=int, default=5000)
    a = a.parse_args()
    model = RandomModel(a.vocab, 256, layers=2, heads=a.heads, d=a.dim)
    layout = S.Layout(a.heads, a.dim, 0, np.full(a.heads, a.bits, np.uint8), np.ones(a.heads * a.dim, np.float32),
                      S.ROW_SCALES_REFIT)
    g = np.random.default_rng(0)
    prompts = [g.integers(1, a.vocab, size=int(n)).tolist() for n in g.integers(1, 300, size=a.batch)]
    sequences, scores = BeamGenerator(model, a.batch, a.beams, layout).run(prompts, a.steps)
    torch.cuda.synchronize()
    for b in range(a.batch):
        print(f"prompt of {len(prompts[b])} tokens")
        for s, t in zip(scores[b].tolist(), sequences[b].tolist()):
            print(f"  {s:9.4f}  {' '.join(map(str, t))}")


if __name__ == "__main__":
    main()
