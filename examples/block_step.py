"""The operators around the projections, used together.

A piece of a decoder block is trained to imitate another one: queries and keys
come from two POET-X projections (packed factors trained, weights frozen),
every head is normalised and rotated in one pass, and a frozen MLP with
trained biases is added to the residual stream.  One step is

    build, q and k projections  ->  norm + rotary of q and k
    up projection, bias, SiLU   ->  down projection, bias, residual
    backward of all of it       ->  clip of the global gradient norm and Adam

Afterwards the factors are merged into the weights, and the merged projection
gives the same queries for a single token.

    python examples/block_step.py [--steps 60]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from orthogonal_reparameterized_packed_gb300 import poetx_packed_size  # noqa: E402
from orthogonal_reparameterized_packed_gb300.block import (PoetxLinear,  # noqa: E402
                                                           PoetxQKNormRope, rope_tables)
from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam, PoetxLayer  # noqa: E402

DIM, HIDDEN, HEAD, HQ, HK = 512, 1024, 64, 8, 4
BLOCK, ORDER, TOKENS = 64, 3, 384


class Piece:
    """Queries, keys and the MLP of one block, with every buffer they need."""

    def __init__(self, weights, tokens, lr=2e-3):
        self.w = weights
        self.q = PoetxLayer(DIM, HQ * HEAD, BLOCK, ORDER, tokens)
        self.k = PoetxLayer(DIM, HK * HEAD, BLOCK, ORDER, tokens)
        self.norm = PoetxQKNormRope(HQ, HK, HEAD, tokens, backward=True)
        self.up = PoetxLinear(DIM, HIDDEN, tokens, act="silu", save_z=True, backward=True)
        self.down = PoetxLinear(HIDDEN, DIM, tokens, backward=True)
        self.cos, self.sin = rope_tables(tokens, HEAD)

        def packed(d):
            return torch.zeros((d // BLOCK, poetx_packed_size(d, BLOCK) // (d // BLOCK)),
                               device="cuda")

        self.theta = {n: (packed(DIM), packed(d)) for n, d in (("q", HQ * HEAD), ("k", HK * HEAD))}
        self.gamma = [torch.ones(HEAD, device="cuda") for _ in range(2)]
        self.bias = [torch.zeros(HIDDEN, device="cuda"), torch.zeros(DIM, device="cuda")]
        self.params = [*self.theta["q"], *self.theta["k"], *self.gamma, *self.bias]
        self.opt = PoetxAdam(self.params, lr=lr)

    def forward(self, x):
        self.x = x
        for n, layer in (("q", self.q), ("k", self.k)):
            layer.build(*self.theta[n])
            layer.forward(x, self.w[n])
        qk = self.norm.forward(self.q.y, self.k.y, *self.gamma, self.cos, self.sin)
        self.hidden = self.up.forward(x, self.w["up"], self.bias[0])
        return (*qk, self.down.forward(self.hidden, self.w["down"], self.bias[1], residual=x))

    def backward(self, dq_out, dk_out, dout):
        dq, dk, dgq, dgk = self.norm.backward(dq_out, dk_out, self.q.y, self.k.y, *self.gamma,
                                              self.cos, self.sin)
        grads = []
        for n, layer, dy in (("q", self.q, dq), ("k", self.k, dk)):
            _, dP, dR = layer.backward(dy, self.x, self.w[n], *self.theta[n])
            grads += [dP, dR]
        dhidden, dbias1 = self.down.backward(dout, self.w["down"])
        _, dbias0 = self.up.backward(dhidden, self.w["up"])
        return grads + [dgq, dgk, dbias0, dbias1]

    def step(self, x, targets, max_norm):
        """(loss, gradient norm before the clip), both on the GPU."""
        outs = self.forward(x)
        diffs = [(o.float() - t.float()) for o, t in zip(outs, targets)]
        loss = sum(0.5 * d.square().mean() for d in diffs)
        grads = self.backward(*[(d / d.numel()).bfloat16() for d in diffs])
        self.opt.step(grads, max_norm=max_norm)
        return loss, self.opt.norm


def main(steps=60, seed=0, quiet=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    weights = {n: normal(o, i, scale=i ** -0.5).bfloat16()
               for n, (i, o) in {"q": (DIM, HQ * HEAD), "k": (DIM, HK * HEAD),
                                 "up": (DIM, HIDDEN), "down": (HIDDEN, DIM)}.items()}
    teacher, student = Piece(weights, TOKENS), Piece(weights, TOKENS)
    for p in teacher.params:
        p += normal(*p.shape, scale=0.03)
    x = normal(TOKENS, DIM).bfloat16()
    targets = [t.clone() for t in teacher.forward(x)]
    losses = []
    for i in range(steps):
        loss, norm = student.step(x, targets, max_norm=0.01)
        losses.append(float(loss))
        if not quiet and i % 10 == 0:
            print(f"step {i:3d}  loss {losses[-1]:.5f}  gradient norm {float(norm):.4f}")

    # serve: the q projection merged into its weight, one token
    before = student.forward(x)[0][:1].clone()
    wq = weights["q"].clone()
    student.q.merge(wq, *student.theta["q"])
    q1 = PoetxLinear(DIM, HQ * HEAD, 1).forward(x[:1], wq)
    one = PoetxQKNormRope(HQ, 0, HEAD, 1)
    served, _ = one.forward(q1, q1[:, :0], student.gamma[0], None, student.cos, student.sin)
    off = float((served.float() - before.float()).norm() / before.float().norm())
    if not quiet:
        print(f"last loss {losses[-1]:.5f}; merged, one token: off by {off:.4f}")
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)
