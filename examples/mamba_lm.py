"""A small Mamba language model on the scan, the layer operators and the block operators: trained on padded
sequences, then decoded token by token.

    python examples/mamba_lm.py [--steps 150] [--dim 128] [--layers 2]

Each block is  t += scale * out_proj(gated_norm(ssm(conv(x)), z)),  x, z = in_proj(norm(t)), with the residual
stream t carried through the norms (``rms_norm(h, residual=t, scale=...)`` scales, adds, stores and normalises in
one pass). In training and over a prompt the convolution hands its result to the scan in the scan's own layout;
a prompt leaves the states of convolution and scan, from which ``block_step`` goes on, one token a call. The
embedding is also the output matrix, against which ``linear_cross_entropy`` takes the loss without logits; padded
targets are -100.

The task is synthetic: each sequence counts up from a random token by a random step, modulo the vocabulary, so the
next token is certain once two have been seen.
"""

import argparse
import math
import os
import sys
import time

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_29_amd import block, layers, scan  # noqa: E402


def weight(*shape):
    return nn.Parameter((torch.randn(shape) / shape[-1] ** 0.5).bfloat16())


class Block(nn.Module):
    def __init__(self, dim, depth, dstate=16, width=4):
        super().__init__()
        inner, rank = 2 * dim, max(1, dim // 16)
        self.scale = 1 / math.sqrt(depth)  # of what a block adds to the residual stream
        self.norm, self.out_norm = nn.Parameter(torch.ones(dim)), nn.Parameter(torch.ones(inner))
        self.w_in, self.w_out = weight(2 * inner, dim), weight(dim, inner)
        bound = width ** -0.5
        self.conv_w = nn.Parameter(torch.empty(inner, 1, width).uniform_(-bound, bound))
        self.conv_b = nn.Parameter(torch.empty(inner).uniform_(-bound, bound))
        self.w_x, self.w_dt = weight(rank + 2 * dstate, inner), weight(inner, rank)
        # softplus(dt_bias) from 0.001 to 0.1, spread over its logarithm
        dt = torch.exp(torch.empty(inner).uniform_(math.log(1e-3), math.log(1e-1)))
        self.dt_bias = nn.Parameter(torch.log(torch.expm1(dt)))
        self.A_log = nn.Parameter(torch.log(torch.arange(1, dstate + 1).float()).repeat(inner, 1))
        self.D = nn.Parameter(torch.ones(inner))

    def new_state(self, batch):
        """The convolution's last inputs and the scan's state, of zeros."""
        inner, dstate = self.A_log.shape
        return (torch.zeros(batch, self.conv_w.shape[2] - 1, inner, dtype=torch.bfloat16, device=self.D.device),
                torch.zeros(batch, inner, dstate, device=self.D.device))

    def forward(self, h, t, state=None):
        """What the block adds to the residual stream, and the stream (h where there is none yet)."""
        if t is None:
            y, t = block.rms_norm(h, self.norm), h
        else:
            y, t = block.rms_norm(h, self.norm, residual=t, scale=self.scale)
        x, z = F.linear(y, self.w_in).chunk(2, -1)  # read in place, as slices
        A = -torch.exp(self.A_log)
        if state is not None and h.shape[1] == 1:
            s = block.block_step(x[:, 0], *state, self.conv_w, self.conv_b, self.w_x, self.w_dt, self.dt_bias, A, D=self.D)[:, None]
        else:
            s = self.sequence(x, A, state)
        return F.linear(block.gated_rms_norm(s.to(z.dtype), z, self.out_norm), self.w_out), t

    def sequence(self, x, A, state):
        if state is None:
            u = block.causal_conv(x, self.conv_w, self.conv_b, scan_layout=True)
        else:
            u, _ = block.causal_conv_fn(x, self.conv_w, self.conv_b, initial_state=state[0], scan_layout=True,
                                        return_last_state=True, last_state_out=state[0])
        rank, dstate = self.w_dt.shape[1], A.shape[1]
        dt, B, C = F.linear(u.contiguous(), self.w_x).split([rank, dstate, dstate], -1)
        delta = F.linear(dt, self.w_dt)
        rows = lambda v: v.transpose(1, 2).contiguous()  # noqa: E731
        args = (u.transpose(1, 2), rows(delta), A, rows(B), rows(C))
        kw = dict(D=self.D, delta_bias=self.dt_bias, delta_softplus=True)
        if state is None:
            y = scan.selective_scan(*args, **kw)
        else:
            y, last = scan.selective_scan_fn(*args, **kw, h0=state[1], return_last_state=True)
            state[1].copy_(last)
        return y.transpose(1, 2)


class MambaLM(nn.Module):
    def __init__(self, vocab, dim, depth):
        super().__init__()
        self.embed = weight(vocab, dim)
        self.blocks = nn.ModuleList(Block(dim, depth) for _ in range(depth))
        self.norm = nn.Parameter(torch.ones(dim))

    def hidden(self, ids, states=None):
        """The normed hidden states of (batch, len) ids; with ``states`` (updated in place) the ids continue what
        the states have seen."""
        h, t = layers.embedding(ids, self.embed, self.embed.shape[1] ** 0.5), None
        for k, b in enumerate(self.blocks):
            h, t = b(h, t, None if states is None else states[k])
        return block.rms_norm(h, self.norm, residual=t, scale=self.blocks[0].scale)[0]

    def new_states(self, batch):
        return [b.new_state(batch) for b in self.blocks]

    def loss(self, ids, target):
        """Mean negative log-likelihood of the targets inside the vocabulary."""
        return block.linear_cross_entropy(self.hidden(ids), self.embed, target)


def sequences(batch, length, vocab, device, generator=None):
    """Counting sequences of different lengths, padded: ids and the next tokens, -100 where there is none."""
    r = lambda *s: torch.rand(*s, generator=generator)  # noqa: E731
    first, step = (r(batch, 1) * vocab).long(), 1 + (r(batch, 1) * 7).long()
    count = (first + step * torch.arange(length + 1)) % vocab
    inside = torch.arange(length) < (length // 2 + (r(batch, 1) * (length // 2 + 1)).long())
    ids = torch.where(inside, count[:, :-1], -1)  # an id outside the vocabulary embeds as zeros
    return ids.to(device), torch.where(inside, count[:, 1:], -100).to(device)


class Decoder:
    """Greedy decoding of ``batch`` rows: the step from one token to the next as a replayed HIP graph."""

    def __init__(self, model, batch):
        self.model, self.states = model, model.new_states(batch)
        self.ids = torch.zeros(batch, 1, dtype=torch.int64, device=model.embed.device)
        self.graph = None

    def kept(self):
        return [*(t for s in self.states for t in s), self.ids]

    def next(self, ids):
        """The logits behind the ids, whose largest becomes the next one."""
        logits = F.linear(self.model.hidden(ids, self.states)[:, -1], self.model.embed)
        self.ids.copy_(logits.argmax(-1, keepdim=True))
        return logits

    @torch.no_grad()
    def step(self):
        self.logits = self.next(self.ids)

    def capture(self):
        """Record ``step``; the states and ids that warming up changes are put back."""
        kept = [t.clone() for t in self.kept()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        for t, k in zip(self.kept(), kept):
            t.copy_(k)

    @torch.no_grad()
    def prompt(self, ids):
        for s in self.kept()[:-1]:
            s.zero_()
        self.next(ids)

    def generate(self, n):
        out = []
        for _ in range(n):
            out.append(self.ids.clone())
            self.graph.replay() if self.graph else self.step()
        return torch.cat(out, 1)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=150)
    p.add_argument("--dim", type=int, default=128)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--vocab", type=int, default=128)
    a = p.parse_args()
    torch.manual_seed(0)
    model = MambaLM(a.vocab, a.dim, a.layers).cuda()
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    for step in range(a.steps):
        loss = model.loss(*sequences(32, 128, a.vocab, "cuda"))
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        if step % 25 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {loss.item():.3f}", flush=True)

    batch, n = 8, 60
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
