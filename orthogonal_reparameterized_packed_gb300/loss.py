"""The losses at the output head, from the last hidden states and the head's weight:
cross entropy and distillation from a teacher's top logits.  bf16 losses alone keep no
logit, gradients one block of tokens' softmax terms (as many bytes as its logits in
bf16; fp32 its logits, and two and a half times those for gradients).  Each class holds
the output buffers and the workspace of one head and enqueues its calls on a stream (the
current one by default); calls of one object on several streams, or of graphs captured
with it, have to be ordered by the caller."""

from __future__ import annotations

import torch

from . import (BF16, F32, GRAD_W, GRAD_X, _check, _stream, load_library,
               poetx_cross_entropy_workspace_size, poetx_distill_workspace_size)
from .block import _address, _need
from .layer import _TORCH_DTYPE, dtype_code

_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}
_LOGITS = {torch.float32: F32, torch.bfloat16: BF16}


class _HeadLoss:
    """Buffers of a head of `vocab` x `d` for up to `tokens` tokens at a time.

    backward: a buffer for dx; weight_grad: one for dW too (a head that is not
    frozen).  block_tokens: how many tokens' terms the workspace holds at a time
    (None: as many as fit 2 GiB).  Fewer take less memory for them, but bf16 heads with
    weight_grad and more than one block also an fp32 dW, 4 vocab d bytes, in the
    workspace: less in all only where the terms saved are more than that."""

    def __init__(self, d, vocab, tokens, top, dtype, device, backward, weight_grad,
                 block_tokens):
        if weight_grad and not backward:
            raise ValueError("weight_grad goes with backward")
        self.d, self.vocab, self.tokens, self.top = d, vocab, tokens, top
        self.block_tokens = 0 if block_tokens is None else block_tokens
        if self.block_tokens < 0 or block_tokens == 0:
            raise ValueError("block_tokens: a number of tokens from 1 on is needed")
        self.code = dtype_code(dtype)
        self.dtype = _TORCH_DTYPE[self.code]
        if tokens < 0 or self._workspace_size(0, max(tokens, 1)) == 0:
            raise ValueError(f"a head of {vocab} x {d} for {tokens} tokens with {top} entries each "
                             "is outside the limits")
        ws = max(self._workspace_size(GRAD_X * bool(backward) + GRAD_W * bool(weight_grad), tokens),
                 self._workspace_size(0, tokens), 16)
        dev = torch.device(device)
        self.loss = torch.empty((tokens,), dtype=torch.float32, device=dev)
        self.total = torch.empty((), dtype=torch.float32, device=dev)
        self.dx = torch.empty((tokens, d), dtype=self.dtype, device=dev) if backward else None
        self.dW = torch.empty((vocab, d), dtype=self.dtype, device=dev) if weight_grad else None
        self.workspace = torch.empty((ws,), dtype=torch.uint8, device=dev)
        self._device = self.loss.get_device()

    def _take(self, x, W, weights, *rest):
        """(tokens, addresses of x, W and weights) after the checks that both losses make."""
        t = x.shape[0]
        if t > self.tokens:
            raise ValueError(f"{t} tokens: the head holds buffers for {self.tokens}")
        at = (_need(x, (t, self.d), self.dtype, "x"),
              _need(W, (self.vocab, self.d), self.dtype, "W"),
              None if weights is None else _need(weights, (t,), torch.float32, "weights"))
        for v in (x, W, *rest) if weights is None else (x, W, weights, *rest):
            if v.get_device() != self._device:
                raise ValueError(f"tensors on {self.loss.device} are needed, got one on {v.device}")
        if self._device >= 0 and torch.cuda.current_device() != self._device:
            raise ValueError(f"the current device has to be {self.loss.device}")
        return t, at

    @staticmethod
    def _indices(v, shape, name):
        """(address, bytes of an index)"""
        if v.dtype not in _INDEX_BYTES:
            raise ValueError(f"{name}: int32 or int64 is needed, got {v.dtype}")
        return _need(v, shape, v.dtype, name), _INDEX_BYTES[v.dtype]

    def _gradients(self):
        if self.dx is None:
            raise RuntimeError(f"{type(self).__name__} was made without backward=True")
        return self.dx.data_ptr(), _address(self.dW)

    def _cut(self, buf, t):
        return buf if t == self.tokens else buf[:t]


class PoetxCrossEntropy(_HeadLoss):
    """Softmax cross entropy of the head's logits x W^T, a target per token.

    targets: int32 or int64; a negative one (e.g. -100) is a token that does not
    count.  weights: the tokens' weights in self.total and in the gradients, float32,
    by default 1 / (tokens that count), so that self.total is their mean."""

    def __init__(self, d, vocab, tokens, dtype="bf16", device="cuda", backward=False,
                 weight_grad=False, block_tokens=None):
        super().__init__(d, vocab, tokens, 1, dtype, device, backward, weight_grad, block_tokens)
        self._call = load_library().poetx_cross_entropy

    def _workspace_size(self, gradients, tokens):
        return poetx_cross_entropy_workspace_size(self.d, self.vocab, tokens, self.code, gradients,
                                                  self.block_tokens)

    def _run(self, x, W, targets, weights, dx, dW, stream):
        t, (x_at, w_at, weights_at) = self._take(x, W, weights, targets)
        idx, size = self._indices(targets, (t,), "targets")
        _check("poetx_cross_entropy", self._call(
            x_at, w_at, idx, size, weights_at, self.loss.data_ptr(), self.total.data_ptr(), dx,
            dW, self.d, self.vocab, t, self.code, self.block_tokens, self.workspace.data_ptr(),
            self.workspace.numel(), _stream(stream)))
        return t

    def forward(self, x, W, targets, weights=None, stream=None):
        """The loss of every token, 0 where none counts (a view of the head's buffer);
        self.total: their weighted sum."""
        return self._cut(self.loss, self._run(x, W, targets, weights, None, None, stream))

    def step(self, x, W, targets, weights=None, stream=None):
        """(loss, dx, dW): the losses and the gradients of self.total; dW None without
        weight_grad."""
        t = self._run(x, W, targets, weights, *self._gradients(), stream)
        return self._cut(self.loss, t), self._cut(self.dx, t), self.dW


class PoetxDistill(_HeadLoss):
    """Distillation from a teacher's `top` largest logits of every token at a
    temperature: temperature^2 times the divergence of the student's softmax over the
    whole vocabulary from the teacher's over its top logits.

    top_indices: int32 or int64, a negative one is no entry (its logit is not used);
    a token without any does not count.  top_logits: float32 or bfloat16, before the
    temperature.  weights as in PoetxCrossEntropy."""

    def __init__(self, d, vocab, tokens, top, temperature=1.0, dtype="bf16", device="cuda",
                 backward=False, weight_grad=False, block_tokens=None):
        if not 1 / 64 <= temperature <= 64:
            raise ValueError(f"temperature: 1/64 to 64 is needed, got {temperature}")
        self.temperature = temperature
        super().__init__(d, vocab, tokens, top, dtype, device, backward, weight_grad,
                         block_tokens)
        self._call = load_library().poetx_distill

    def _workspace_size(self, gradients, tokens):
        return poetx_distill_workspace_size(self.d, self.vocab, tokens, self.top, self.code,
                                            gradients, self.block_tokens)

    def _run(self, x, W, top_indices, top_logits, weights, dx, dW, stream):
        t, (x_at, w_at, weights_at) = self._take(x, W, weights, top_indices, top_logits)
        idx, size = self._indices(top_indices, (t, self.top), "top_indices")
        if top_logits.dtype not in _LOGITS:
            raise ValueError(f"top_logits: float32 or bfloat16 is needed, got {top_logits.dtype}")
        logits = _need(top_logits, (t, self.top), top_logits.dtype, "top_logits")
        _check("poetx_distill", self._call(
            x_at, w_at, idx, size, logits, _LOGITS[top_logits.dtype], weights_at,
            self.loss.data_ptr(), self.total.data_ptr(), dx, dW, self.d, self.vocab, t, self.top,
            self.temperature, self.code, self.block_tokens, self.workspace.data_ptr(),
            self.workspace.numel(), _stream(stream)))
        return t

    def forward(self, x, W, top_indices, top_logits, weights=None, stream=None):
        """As PoetxCrossEntropy.forward."""
        return self._cut(self.loss,
                         self._run(x, W, top_indices, top_logits, weights, None, None, stream))

    def step(self, x, W, top_indices, top_logits, weights=None, stream=None):
        """As PoetxCrossEntropy.step."""
        t = self._run(x, W, top_indices, top_logits, weights, *self._gradients(), stream)
        return self._cut(self.loss, t), self._cut(self.dx, t), self.dW
