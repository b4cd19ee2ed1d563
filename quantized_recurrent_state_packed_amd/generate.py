"""Beam search with a small random linear-attention model, from ragged prompts to
sequences: every state-related step runs in the library.

    prompts --stepq_linear_prefill--> states --stepq_pack--> one slot a request
    last logits --stepq_beam_select--> tokens, parents --stepq_beam_reorder--> a slot a beam
    tokens --stepq_decode_step on the packed slots--> logits --select, reorder--> ...

    python -m quantized_recurrent_state_packed_amd.generate --bits 6 --beams 4 --steps 16

The model (embedding, per layer q, k, v, beta, gate and output projections,
logits) has random weights and stands in for whatever computes q, k, v from tokens.

With --drafts K, speculative sampling with a random model of gated recurrent blocks, whose first layers
draft K tokens at a time that all of them verify:

    prompts --stepq_scan_forward, stepq_norm_forward--> states of both models
    draft: --stepq_scan_step--> logits --stepq_verify_drafts without drafts--> a token, K times
    target: the K + 1 tokens at once --stepq_scan_forward on a copy of the states--> logits
    --stepq_verify_drafts--> accepted tokens and the next one --stepq_scan_forward--> states behind them

    python -m quantized_recurrent_state_packed_amd.generate --drafts 4 --steps 16
"""
from __future__ import annotations

import argparse

import numpy as np

from . import beam
from . import stepq as S
from .draft import DraftVerify
from .linear import LinearAttention
from .norm import BlockNorm
from .recurrence import GatedRecurrence


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


class RecurrentModel:
    """A language model of gated recurrent blocks with random weights: per layer the recurrence between
    projections, then norm, gate, residual sum and the next layer's norm in one pass."""

    def __init__(self, vocab: int, width: int, layers: int, seed: int = 0, device="cuda"):
        import torch
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale, shift=0.0):
            return (shift + torch.randn(*shape, generator=g) * scale).to(device)

        self.vocab, self.width, self.layers, self.device = vocab, width, layers, device
        self.embedding = weight(vocab, width, scale=1.0)
        self.first = weight(width, scale=0.1, shift=1.0)
        self.inner = [weight(width, 4 * width, scale=width ** -0.5) for _ in range(layers)]     # x, gate_a, gate_x, gate
        self.decay = [weight(width, scale=1.5, shift=-4.0) for _ in range(layers)]
        self.post = [weight(width, scale=0.1, shift=1.0) for _ in range(layers)]
        self.scale = [weight(width, scale=0.05, shift=0.7) for _ in range(layers)]
        self.pre = [weight(width, scale=0.1, shift=1.0) for _ in range(layers)]
        self.head = weight(width, vocab, scale=2.0 * width ** -0.5)
        self.recurrence = GatedRecurrence(width)
        self.opening = BlockNorm(width, post=False)
        self.norm = BlockNorm(width)

    def first_layers(self, layers: int):
        """A model of this one's first layers, with the same embedding, head and weights: a draft of it."""
        import copy
        m = copy.copy(self)
        m.layers = layers
        return m

    def states(self, num_slots: int):
        return [self.recurrence.states(num_slots, device=self.device) for _ in range(self.layers)]

    def _through(self, tokens, recur):
        """Logits of tokens [T]; recur(layer, x, gate_a, gate_x, y) runs the layer's recurrence."""
        import torch
        stream = self.embedding[tokens]
        normed, y = torch.empty_like(stream), torch.empty_like(stream)
        self.opening.forward(stream, None, normed, pre_weight=self.first)
        for n in range(self.layers):
            x, gate_a, gate_x, gate = (normed @ self.inner[n]).view(-1, 4, self.width).unbind(1)
            recur(n, x, gate_a, gate_x, y)
            self.norm.forward(y, stream, normed, gate=gate, residual=stream, post_weight=self.post[n], scale=self.scale[n],
                              pre_weight=self.pre[n])
        return normed @ self.head

    def prefill(self, tokens, cu_seqlens, slots, states, resume=None, workspace=None):
        """Ragged prompts, rows of tokens [T]; rows of no request have logits that mean nothing."""
        def recur(n, x, gate_a, gate_x, y):
            y.zero_()
            self.recurrence.prefill(cu_seqlens, x, gate_a, gate_x, self.decay[n], slots, states[n], y, resume=resume,
                                    workspace=workspace)
        return self._through(tokens, recur)

    def step(self, tokens, slots, states):
        """One token of every request."""
        def recur(n, x, gate_a, gate_x, y):
            self.recurrence.step(slots, x, gate_a, gate_x, self.decay[n], states[n], y)
        return self._through(tokens, recur)


class DraftGenerator:
    """Speculative sampling over a batch of prompts: `drafts` tokens at a time are drawn from the draft model
    and verified by the target model, whose own distribution the result has."""

    def __init__(self, target: RecurrentModel, draft: RecurrentModel, batch: int, drafts: int, temperature: float = 1.0):
        import torch
        if target.vocab != draft.vocab:
            raise S.StepqError(S.STEPQ_ERR_INVALID_ARG, "DraftGenerator", "the models' vocabularies differ")
        if drafts < 1:
            raise S.StepqError(S.STEPQ_ERR_INVALID_ARG, "DraftGenerator", "at least one draft at a time is needed")
        device = target.device
        self.target, self.draft, self.batch, self.drafts, self.device = target, draft, batch, drafts, device
        self.verify = DraftVerify(batch, drafts, target.vocab, device=device)
        self.draw = DraftVerify(batch, 0, target.vocab, device=device)
        self.temperature = torch.full((batch,), float(temperature), device=device)
        self.slots = torch.arange(batch, dtype=torch.int32, device=device)
        self.resume = torch.ones(batch, dtype=torch.uint8, device=device)
        self.rows = torch.arange(batch * (drafts + 1), device=device)
        self.whole = torch.arange(0, batch * (drafts + 1) + 1, drafts + 1, dtype=torch.int32, device=device)
        self.workspaces = [m.recurrence.workspace(batch, batch * (drafts + 1), device=device) for m in (target, draft)]

    def prefill(self, prompts):
        """Prompts (non-empty lists of tokens) but for their last tokens, which are returned; both models' states."""
        import torch
        if len(prompts) != self.batch or any(len(p) == 0 for p in prompts):
            raise S.StepqError(S.STEPQ_ERR_INVALID_ARG, "DraftGenerator", f"{self.batch} non-empty prompts are needed")
        if any(min(p) < 0 or max(p) >= self.target.vocab for p in prompts):
            raise S.StepqError(S.STEPQ_ERR_INVALID_ARG, "DraftGenerator",
                               f"a prompt has tokens outside of the vocabulary of {self.target.vocab}")
        cu = torch.tensor(np.r_[0, np.cumsum([len(p) - 1 for p in prompts])], dtype=torch.int32, device=self.device)
        tokens = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.long, device=self.device)
        self.states = [m.states(self.batch) for m in (self.target, self.draft)]
        for m, states in zip((self.target, self.draft), self.states):
            m.prefill(tokens, cu, self.slots, states)
        return torch.tensor([p[-1] for p in prompts], device=self.device)

    def round(self, last, uniforms):
        """One round from the tokens `last` [batch] that no state has seen yet, with uniforms [batch, 2 drafts + 1]
        (drafting, then verifying): accepted [batch] and tokens [batch, drafts + 1] of the verification."""
        import torch
        b, k = self.batch, self.drafts
        states = [s.clone() for s in self.states[1]]
        tokens, logits = [last], []
        for n in range(k):
            logits.append(self.draft.step(tokens[-1], self.slots, states))
            _, drawn = self.draw(logits[-1], None, uniforms[:, n:n + 1].contiguous(), temperature=self.temperature)
            tokens.append(drawn[:, 0].long())
        tokens = torch.stack(tokens, 1)                                     # [batch, drafts + 1]
        states = [s.clone() for s in self.states[0]]
        ahead = self.target.prefill(tokens.view(-1), self.whole, self.slots, states, resume=self.resume,
                                    workspace=self.workspaces[0])
        accepted, out = self.verify(ahead, tokens[:, 1:].int().contiguous(), uniforms[:, k:].contiguous(),
                                    draft_logits=torch.stack(logits, 1).view(b * k, -1), temperature=self.temperature)
        # the states behind the accepted tokens: `last` and as many drafts, of all requests in a row
        cu = torch.cat([self.whole[:1], (accepted + 1).cumsum(0).int()])
        owner = torch.searchsorted(cu[1:].contiguous(), self.rows.int(), right=True).clamp(max=b - 1)
        source = (owner * (k + 1) + self.rows - cu[owner]).clamp(max=b * (k + 1) - 1)
        kept = tokens.view(-1)[source]
        for m, states, ws in zip((self.target, self.draft), self.states, self.workspaces):
            m.prefill(kept, cu, self.slots, states, resume=self.resume, workspace=ws)
        return accepted.clone(), out.clone()          # the next round overwrites these

    def run(self, prompts, steps: int, seed: int = 0):
        """At least `steps` tokens a request, cut to `steps`: [batch][steps]; and the share of drafts accepted."""
        import torch
        last = self.prefill(prompts)
        gen = torch.Generator(device=self.device).manual_seed(seed)
        sequences, kept, rounds = [[] for _ in range(self.batch)], 0, 0
        while min(len(s) for s in sequences) < steps:
            u = torch.rand(self.batch, 2 * self.drafts + 1, generator=gen, device=self.device)
            accepted, out = self.round(last, u)
            last = out.gather(1, accepted.long()[:, None])[:, 0].long()
            for s, n, row in zip(sequences, accepted.tolist(), out.tolist()):
                s += row[:n + 1]
                kept += n
            rounds += self.batch * self.drafts
        return [s[:steps] for s in sequences], kept / max(1, rounds)


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
    a.add_argument("--drafts", type=int, default=0, help="speculative sampling, so many drafted tokens at a time")
    a.add_argument("--temperature", type=float, default=1.0, help="of speculative sampling; 0: greedy")
    a = a.parse_args()
    g = np.random.default_rng(0)
    prompts = [g.integers(1, a.vocab, size=int(n)).tolist() for n in g.integers(1, 300, size=a.batch)]
    if a.drafts > 0:
        target = RecurrentModel(a.vocab, 256, layers=4)
        sequences, share = DraftGenerator(target, target.first_layers(3), a.batch, a.drafts, a.temperature).run(prompts, a.steps)
        for p, s in zip(prompts, sequences):
            print(f"prompt of {len(p)} tokens\n  {' '.join(map(str, s))}")
        print(f"{share:.2f} of the drafted tokens accepted")
        return
    model = RandomModel(a.vocab, 256, layers=2, heads=a.heads, d=a.dim)
    layout = S.Layout(a.heads, a.dim, 0, np.full(a.heads, a.bits, np.uint8), np.ones(a.heads * a.dim, np.float32),
                      S.ROW_SCALES_REFIT)
    sequences, scores = BeamGenerator(model, a.batch, a.beams, layout).run(prompts, a.steps)
    torch.cuda.synchronize()
    for b in range(a.batch):
        print(f"prompt of {len(prompts[b])} tokens")
        for s, t in zip(scores[b].tolist(), sequences[b].tolist()):
            print(f"  {s:9.4f}  {' '.join(map(str, t))}")


if __name__ == "__main__":
    main()
