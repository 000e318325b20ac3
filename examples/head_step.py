"""The losses at the output head, used together.

A student with one POET-X projection (packed factors trained, weight frozen) and an
output head (trained) learns from data and from a teacher's top logits.  One step is

    build, projection                ->  the last hidden states
    cross entropy, distillation      ->  losses, gradients of both by the hidden
                                         states and by the head's weight
    backward of the projection       ->  clip of the global gradient norm and Adam

Some tokens are padding, and some have no teacher.  Afterwards the factors are merged
into the weight, and single tokens are scored with it.

    python examples/head_step.py [--steps 20]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from orthogonal_reparameterized_packed_gb300 import poetx_packed_size  # noqa: E402
from orthogonal_reparameterized_packed_gb300.block import PoetxLinear  # noqa: E402
from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam, PoetxLayer  # noqa: E402
from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill  # noqa: E402

DIM, VOCAB, TOP, BLOCK, ORDER, TOKENS = 512, 1537, 8, 64, 3, 300
TEMPERATURE, SHARE = 2.0, 0.5  # of the distillation: its temperature and weight


class Student:
    def __init__(self, W0, head, tokens, lr=1e-3):
        self.W0, self.head = W0, head
        self.layer = PoetxLayer(DIM, DIM, BLOCK, ORDER, tokens)
        self.ce = PoetxCrossEntropy(DIM, VOCAB, tokens, backward=True, weight_grad=True)
        self.kd = PoetxDistill(DIM, VOCAB, tokens, top=TOP, temperature=TEMPERATURE,
                               backward=True, weight_grad=True)
        packed = poetx_packed_size(DIM, BLOCK) // (DIM // BLOCK)
        self.theta = [torch.zeros((DIM // BLOCK, packed), device="cuda") for _ in range(2)]
        self.master = head.float()  # the head's weight is trained in float32
        self.opt = PoetxAdam([*self.theta, self.master], lr=lr)

    def gradients(self, x, targets, top_indices, top_logits):
        """(loss, [gradients of theta_P, theta_R and the head])"""
        self.layer.build(*self.theta)
        h = self.layer.forward(x, self.W0)
        _, dh, dhead = self.ce.step(h, self.head, targets)
        _, dh_kd, dhead_kd = self.kd.step(h, self.head, top_indices, top_logits)
        dh = torch.add(dh, dh_kd, alpha=SHARE)
        dhead = torch.add(dhead.float(), dhead_kd, alpha=SHARE)
        _, dP, dR = self.layer.backward(dh, x, self.W0, *self.theta)
        return self.ce.total + SHARE * self.kd.total, [dP, dR, dhead]

    def step(self, *batch):
        loss, grads = self.gradients(*batch)
        self.opt.step([g.view(p.shape) for g, p in zip(grads, self.opt.params)], max_norm=1.0)
        self.head.copy_(self.master)
        return loss


def batch(g, x, teacher_logits):
    """Targets and a teacher's top logits; a tenth of the tokens is padding, another
    tenth has no teacher."""
    targets = torch.distributions.Categorical(logits=teacher_logits).sample()
    top = teacher_logits.topk(TOP, 1)
    indices, logits = top.indices.clone(), top.values.contiguous()
    order = torch.randperm(len(targets), generator=g, device="cuda")
    tenth = len(targets) // 10
    targets[order[:tenth]] = -100
    indices[order[:2 * tenth]] = -1
    return x, targets, indices, logits


def start(seed=0):
    """(student, its batch)"""
    torch.manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    W0 = normal(DIM, DIM, scale=DIM ** -0.5).bfloat16()
    head = normal(VOCAB, DIM, scale=2 * DIM ** -0.5).bfloat16()
    x = normal(TOKENS, DIM).bfloat16()
    teacher = x.float() @ normal(DIM, DIM, scale=DIM ** -0.5).t() @ head.float().t()
    return Student(W0, head.clone(), TOKENS), batch(g, x, teacher)


def main(steps=20, seed=0, quiet=False):
    student, data = start(seed)
    losses = []
    for i in range(steps):
        losses.append(float(student.step(*data)))
        if not quiet and i % 5 == 0:
            print(f"step {i:3d}  loss {losses[-1]:.4f}")
    # serve: the projection merged into its weight, tokens scored one at a time
    x, targets = data[:2]
    student.layer.build(*student.theta)
    h = student.layer.forward(x, student.W0)
    together = student.ce.forward(h, student.head, targets).clone()
    W = student.W0.clone()
    student.layer.merge(W, *student.theta)
    project, score = PoetxLinear(DIM, DIM, 1), PoetxCrossEntropy(DIM, VOCAB, 1)
    off = 0.0
    for t in range(4):
        one = score.forward(project.forward(x[t:t + 1], W), student.head, targets[t:t + 1])
        off = max(off, abs(float(one[0]) - float(together[t])))
    if not quiet:
        print(f"last loss {losses[-1]:.4f}; scores of single tokens are {off:.4f} away at most")
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
