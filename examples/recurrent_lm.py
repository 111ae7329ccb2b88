"""A small recurrent language model on the layer operators: trained on packed sequences, then decoded
token by token.

    python examples/recurrent_lm.py [--steps 150] [--dim 256] [--layers 2]

Each block is  t += mixer(norm(t));  t += down(gated_ffn(norm(t)))  with the residual stream t carried
through the norms (``layer_norm(h, residual=t)`` adds, stores and normalises in one pass). The mixer is
the gated linear recurrence on slices of one projection; documents lie one after another in a row, and
``reset`` keeps a document from seeing the one before it. The embedding is also the output matrix.

Decoding holds one fp32 state per layer and updates it in place, so a token costs the same at any
position; the step is captured into a HIP graph once and replayed.

The task is synthetic: each document counts up from a random token by a random step, modulo the
vocabulary, so the next token is certain once two have been seen.
"""

import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_29_amd import layers  # noqa: E402


def weight(*shape):
    return nn.Parameter((torch.randn(shape) / shape[-1] ** 0.5).bfloat16())


class Norm(nn.Module):
    def __init__(self, dim):
        super().__init__()
        self.weight, self.bias = nn.Parameter(torch.ones(dim)), nn.Parameter(torch.zeros(dim))

    def forward(self, h, t):
        """The norm of h + t, and that sum (h itself where there is no t yet)."""
        if t is None:
            return layers.layer_norm(h, self.weight, self.bias), h
        return layers.layer_norm(h, self.weight, self.bias, residual=t)


class Block(nn.Module):
    def __init__(self, dim, hidden):
        super().__init__()
        self.norm1, self.norm2 = Norm(dim), Norm(dim)
        self.w_in, self.w_out = weight(4 * dim, dim), weight(dim, dim)
        # a = exp(-8 softplus(lam) sigmoid(r)): about 0.9 to 0.999 a step at an open gate
        self.lam = nn.Parameter(torch.log(torch.expm1(-torch.log(torch.empty(dim).uniform_(0.9, 0.999)) / 8)))
        self.w_gate, self.w_up, self.w_down = weight(hidden, dim), weight(hidden, dim), weight(dim, hidden)

    def forward(self, h, t, reset=None, state=None):
        y, t = self.norm1(h, t)
        x, r, i, z = F.linear(y, self.w_in).chunk(4, -1)  # read in place, as slices
        if state is None:
            s = layers.gated_scan(x, r, i, self.lam, reset=reset)
        else:
            s, _ = layers.gated_scan_fn(x, r, i, self.lam, h0=state, return_last_state=True, last_state_out=state)
        h = F.linear(s * F.silu(z), self.w_out)
        y, t = self.norm2(h, t)
        return F.linear(layers.gated_ffn(y, self.w_gate, self.w_up), self.w_down), t


class RecurrentLM(nn.Module):
    def __init__(self, vocab, dim, depth, hidden):
        super().__init__()
        self.embed = weight(vocab, dim)
        self.blocks = nn.ModuleList(Block(dim, hidden) for _ in range(depth))
        self.norm = Norm(dim)

    def forward(self, ids, reset=None, states=None):
        """Logits of (batch, len) ids; with ``states`` (one (batch, dim) fp32 tensor a layer, updated in
        place) the ids continue what the states have seen."""
        h, t = layers.embedding(ids, self.embed, self.embed.shape[1] ** 0.5), None
        for k, block in enumerate(self.blocks):
            h, t = block(h, t, reset, None if states is None else states[k])
        return F.linear(self.norm(h, t)[0], self.embed)

    def new_states(self, batch):
        return [torch.zeros(batch, self.embed.shape[1], device=self.embed.device) for _ in self.blocks]

    def loss(self, ids, reset):
        """Mean negative log-likelihood of each next token of the same document."""
        logits = self(ids, reset)[:, :-1].float()
        target = ids[:, 1:].masked_fill(reset[:, 1:], -100)
        return F.cross_entropy(logits.flatten(0, 1), target.flatten(), ignore_index=-100)


def documents(batch, length, vocab, device, generator=None):
    """Packed counting documents: ids (batch, length) and the resets at their first tokens."""
    r = lambda *s: torch.rand(*s, generator=generator)  # noqa: E731
    reset = r(batch, length) < 1 / 40
    reset[:, 0] = True
    first, step = (r(batch, length) * vocab).long(), 1 + (r(batch, length) * 7).long()
    at = torch.where(reset, torch.arange(length).expand(batch, length), 0).cummax(1).values  # where the document begins
    ids = (first.gather(1, at) + step.gather(1, at) * (torch.arange(length) - at)) % vocab
    return ids.to(device), reset.to(device)


class Decoder:
    """Greedy decoding of ``batch`` rows: the step from one token to the next as a replayed HIP graph."""

    def __init__(self, model, batch):
        self.model, self.states = model, model.new_states(batch)
        self.ids = torch.zeros(batch, 1, dtype=torch.int64, device=model.embed.device)
        self.graph = None

    @torch.no_grad()
    def step(self):
        self.logits = self.model(self.ids, states=self.states)[:, -1]
        self.ids.copy_(self.logits.argmax(-1, keepdim=True))

    def capture(self):
        """Record ``step``; the states and ids that warming up changes are put back."""
        kept = [t.clone() for t in (*self.states, self.ids)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        for t, k in zip((*self.states, self.ids), kept):
            t.copy_(k)

    @torch.no_grad()
    def prompt(self, ids):
        for s in self.states:
            s.zero_()
        logits = self.model(ids, states=self.states)[:, -1]
        self.ids.copy_(logits.argmax(-1, keepdim=True))

    def generate(self, n):
        out = []
        for _ in range(n):
            out.append(self.ids.clone())
            self.graph.replay() if self.graph else self.step()
        return torch.cat(out, 1)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=150)
    p.add_argument("--dim", type=int, default=256)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--vocab", type=int, default=128)
    a = p.parse_args()
    torch.manual_seed(0)
    model = RecurrentLM(a.vocab, a.dim, a.layers, 2 * a.dim + 88).cuda()
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    for step in range(a.steps):
        ids, reset = documents(16, 512, a.vocab, "cuda")
        loss = model.loss(ids, reset)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        if step % 25 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {loss.item():.3f}", flush=True)

    batch, n = 8, 100
    first, stride = torch.randint(a.vocab, (batch, 1)), torch.randint(1, 8, (batch, 1))
    count = ((first + stride * torch.arange(20 + n)) % a.vocab).cuda()
    decoder = Decoder(model, batch)
    decoder.capture()
    decoder.prompt(count[:, :20])
    torch.cuda.synchronize()
    begin = time.perf_counter()
    got = decoder.generate(n)
    torch.cuda.synchronize()
    each = (time.perf_counter() - begin) / n
    right = (got == count[:, 20:]).float().mean().item()
    print(f"decoded {batch} x {n} tokens, {100 * right:.1f}% as counted, {1e6 * each:.0f} us a step")


if __name__ == "__main__":
    main()
