"""A small selective state space model trained and sampled with the package's
layer operators: block norm -> input projection -> causal convolution ->
selective scan -> output projection -> block norm.

Training runs the prompt forms and their gradients (the autograd functions);
generation carries the convolution's and the scan's states from the prompt
into the single-token forms.  The projections are plain matrix products.

    python examples/selective_model.py [--steps 150]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_sequence_cumsum_gb300 as ssd  # noqa: E402


class Layer(torch.nn.Module):
    """Projections, convolution and scan of one block; dim -> dim."""

    def __init__(self, dim, inner, dstate, rank, width):
        super().__init__()
        self.inner, self.dstate, self.rank = inner, dstate, rank

        def weight(*shape):
            return torch.nn.Parameter(torch.randn(shape) / math.sqrt(shape[0]))
        self.w_in, self.w_x = weight(dim, 2 * inner), weight(inner, rank + 2 * dstate)
        self.w_dt, self.w_out = weight(rank, inner), weight(inner, dim)
        self.conv = torch.nn.Parameter((torch.rand(inner, width) * 2 - 1) / math.sqrt(width))
        self.conv_bias = torch.nn.Parameter(torch.zeros(inner))
        self.log_a = torch.nn.Parameter(torch.log(torch.arange(1.0, dstate + 1)).repeat(inner, 1))
        self.skip = torch.nn.Parameter(torch.ones(inner))
        # softplus(dt_bias) between 1e-3 and 1e-1
        self.dt_bias = torch.nn.Parameter(torch.log(torch.expm1(torch.exp(
            torch.empty(inner).uniform_(math.log(1e-3), math.log(1e-1))))))

    def inputs(self, x):
        """u and z, two slices of one projection."""
        return (x @ self.w_in.to(x.dtype)).split(self.inner, -1)

    def steps(self, u):
        """dt, B and C of each token."""
        r, B, C = (u @ self.w_x.to(u.dtype)).split((self.rank, self.dstate, self.dstate), -1)
        return r @ self.w_dt.to(u.dtype), B, C

    def forward(self, x):
        """A prompt [batch, seqlen, dim]; returns the output and the two states."""
        u, z = self.inputs(x)
        u, conv_state = ssd.CausalConvFunction.apply(u, self.conv, self.conv_bias)
        dt, B, C = self.steps(u)
        y, state = ssd.SelectiveScanFunction.apply(u, dt, -torch.exp(self.log_a), B, C, self.skip, z, self.dt_bias)
        return y @ self.w_out.to(x.dtype), (conv_state, state)

    def token(self, x, states):
        """One token [batch, dim]; updates the states in place."""
        u, z = self.inputs(x)
        u, _ = ssd.ssd_causal_conv_step(u, self.conv, states[0], self.conv_bias)
        dt, B, C = self.steps(u)
        y, _ = ssd.ssd_selective_scan_step(u, dt, -torch.exp(self.log_a), B, C, self.skip, states[1], z, self.dt_bias)
        return y @ self.w_out.to(x.dtype)


class Model(torch.nn.Module):
    def __init__(self, vocab=64, dim=128, inner=256, dstate=16, rank=8, width=4, layers=2):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(vocab, dim) / math.sqrt(dim))
        self.layers = torch.nn.ModuleList(Layer(dim, inner, dstate, rank, width) for _ in range(layers))
        # norm before each block (and the last one's output), after it, and its gate
        self.norm = torch.nn.ParameterList(torch.ones(dim) for _ in range(layers + 1))
        self.post = torch.nn.ParameterList(torch.ones(dim) for _ in range(layers))
        self.gate = torch.nn.ParameterList(torch.ones(1, dim) for _ in range(layers))
        self.scale = 1.0 / math.sqrt(2 * layers)

    def between(self, i, y, residual):
        """The norms around block i's output (i = 0: only the first block's input)."""
        post, gate = (self.post[i - 1], self.gate[i - 1]) if i else (None, None)
        return ssd.BlockNormFunction.apply(y.contiguous(), residual, self.norm[i], post, gate,
                                           self.scale if i else 1.0)

    def run(self, tokens, block):
        x, residual = self.between(0, self.embed.bfloat16()[tokens], None)
        for i, layer in enumerate(self.layers):
            x, residual = self.between(i + 1, block(i, layer, x), residual)
        return (x @ self.embed.bfloat16().t()).float()

    def forward(self, tokens):
        """Logits of a prompt and the layers' states after it."""
        states = []

        def block(i, layer, x):
            y, s = layer(x)
            states.append(s)
            return y
        return self.run(tokens, block), states

    def token(self, tokens, states):
        """Logits of one token per sequence; the states move on by it."""
        return self.run(tokens, lambda i, layer, x: layer.token(x, states[i]))


def batch(g, n, length, table):
    """Sequences whose next token is given by the one before the last: a table
    of all tokens, from two random ones."""
    seq = [torch.randint(0, table.numel(), (n,), generator=g, device="cuda") for _ in range(2)]
    while len(seq) < length:
        seq.append(table[seq[-2]])
    return torch.stack(seq, 1)


def main(steps=150, seqlen=96, sequences=16, generate=24, quiet=False):
    torch.manual_seed(0)
    model = Model().cuda()
    vocab = model.embed.shape[0]
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(vocab, generator=g, device="cuda")
    losses = []
    for step in range(steps):
        data = batch(g, sequences, seqlen + 1, table)
        logits, _ = model(data[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.reshape(-1, vocab), data[:, 1:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if not quiet and step % 25 == 0:
            print(f"step {step:3d}  loss {losses[-1]:.3f}")

    with torch.no_grad():
        whole = batch(g, 4, 32 + generate, table)
        prompt = whole[:, :32]
        logits, states = model(prompt)
        tokens, seen = [logits[:, -1].argmax(-1)], [logits[:, -1]]
        for _ in range(generate - 1):
            seen.append(model.token(tokens[-1], states))
            tokens.append(seen[-1].argmax(-1))
        # the same sequences as one prompt
        full, _ = model(torch.cat([prompt, torch.stack(tokens[:-1], 1)], 1))
        gap = float((torch.stack(seen, 1) - full[:, 31:]).abs().max() / full.abs().max())
        right = float((torch.stack(tokens, 1) == whole[:, 32:]).float().mean())
    if not quiet:
        print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; {generate} tokens generated, "
              f"{100 * right:.0f}% as the table has them; token by token against one prompt: {gap:.1e}")
    return losses, gap, right


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=150)
    main(p.parse_args().steps)
