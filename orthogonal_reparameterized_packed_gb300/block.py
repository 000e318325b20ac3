"""What stands around the projections in a decoder block: the matrix product
with bias, activation and residual (for frozen or merged weights), the norm of
queries and keys with the rotary embedding, and the clip of the gradients.
Each class holds the output buffers and the workspace of one such step and
enqueues its calls on a stream (the current one by default)."""

from __future__ import annotations

import torch

from . import (ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, poetx_clip_grads,
               poetx_grad_norm, poetx_grad_norm_workspace_size, poetx_linear_backward,
               poetx_linear_backward_workspace_size, poetx_linear_forward,
               poetx_linear_forward_workspace_size, poetx_qk_norm_rope_backward,
               poetx_qk_norm_rope_backward_workspace_size, poetx_qk_norm_rope_forward)
from .layer import _TORCH_DTYPE, dtype_code

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU,
               "gelu_tanh": ACT_GELU_TANH}


def _need(t, shape, dtype, name):
    """t is a contiguous CUDA tensor of this shape and type, or a ValueError."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: a contiguous CUDA tensor of shape {shape} and type {dtype} is "
                         f"needed, got {tuple(t.shape)}, {t.dtype}")


class PoetxLinear:
    """y = act(x W^T + bias) + residual for up to `tokens` tokens at a time,
    W [d_out][d_in] frozen (e.g. merged by PoetxLayer.merge).

    save_z: the forward keeps z = x W^T + bias, which the backward of an
    activation needs; backward: buffers for the gradients dx and dbias."""

    def __init__(self, d_in, d_out, tokens, act="none", dtype="bf16", device="cuda",
                 save_z=False, backward=False):
        self.d_in, self.d_out, self.tokens = d_in, d_out, tokens
        self.act, self.code = ACTIVATIONS[act], dtype_code(dtype)
        self.dtype = _TORCH_DTYPE[self.code]
        dev = torch.device(device)
        self.y = torch.empty((tokens, d_out), dtype=self.dtype, device=dev)
        self.z = torch.empty((tokens, d_out), dtype=self.dtype, device=dev) if save_z else None
        self.dx = self.dbias = None
        ws = poetx_linear_forward_workspace_size(d_in, d_out, tokens, self.code)
        if backward:
            self.dx = torch.empty((tokens, d_in), dtype=self.dtype, device=dev)
            self.dbias = torch.empty((d_out,), dtype=torch.float32, device=dev)
            ws = max(ws, poetx_linear_backward_workspace_size(d_in, d_out, tokens, self.act,
                                                              self.code, True))
        self.workspace = torch.empty((max(ws, 16),), dtype=torch.uint8, device=dev)

    def _rows(self, t):
        if t > self.tokens:
            raise ValueError(f"{t} tokens: the layer holds buffers for {self.tokens}")
        return t

    def forward(self, x, W, bias=None, residual=None, stream=None):
        """y for x's tokens (a view of the layer's buffer; so is z, kept in
        self.z's first rows)."""
        t = self._rows(x.shape[0])
        _need(x, (t, self.d_in), self.dtype, "x")
        _need(W, (self.d_out, self.d_in), self.dtype, "W")
        if bias is not None:
            _need(bias, (self.d_out,), torch.float32, "bias")
        if residual is not None:
            _need(residual, (t, self.d_out), self.dtype, "residual")
        poetx_linear_forward(x, W, bias, residual, self.y, self.z, self.d_in, self.d_out, t,
                             self.act, self.code, self.workspace, stream)
        return self.y if t == self.tokens else self.y[:t]

    def backward(self, dy, W, z=None, stream=None):
        """(dx, dbias) from dy and the z of the forward (self.z by default);
        the residual's gradient is dy."""
        if self.dx is None:
            raise RuntimeError("PoetxLinear was made without backward=True")
        t = self._rows(dy.shape[0])
        z = self.z if z is None else z
        _need(dy, (t, self.d_out), self.dtype, "dy")
        _need(W, (self.d_out, self.d_in), self.dtype, "W")
        if self.act != ACT_NONE:
            if z is None:
                raise ValueError("the backward of an activation needs z (save_z=True)")
            _need(z[:t] if z.shape[0] != t else z, (t, self.d_out), self.dtype, "z")
        poetx_linear_backward(dy, z, W, self.dx, self.dbias, self.d_in, self.d_out, t, self.act,
                              self.code, self.workspace, stream)
        return (self.dx if t == self.tokens else self.dx[:t]), self.dbias


def rope_tables(rows, rot_dim, base=10000.0, device="cuda"):
    """(cos, sin) [rows][rot_dim / 2] float32 of the plain rotary embedding,
    angle = position * base^(-2 i / rot_dim), computed in float64."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * (base ** (-i / rot_dim))[None, :]
    return angle.cos().float().to(device), angle.sin().float().to(device)


class PoetxQKNormRope:
    """RMS norm of every query and key head and the rotary embedding, in one
    pass over q and k, for up to `tokens` tokens at a time.

    q, k: [tokens][heads * head_dim] (or [tokens][heads][head_dim]) tensors
    whose last dimensions are contiguous; rows may be strided (slices of a
    fused projection).  cos, sin: [rows][rot_dim / 2] float32 (rope_tables)."""

    def __init__(self, n_q_heads, n_k_heads, head_dim, tokens, rot_dim=None, eps=1e-6,
                 interleaved=False, dtype="bf16", device="cuda", backward=False):
        self.hq, self.hk, self.D, self.tokens = n_q_heads, n_k_heads, head_dim, tokens
        self.rot = head_dim if rot_dim is None else rot_dim
        self.eps, self.interleaved = eps, interleaved
        self.code = dtype_code(dtype)
        self.dtype = _TORCH_DTYPE[self.code]
        dev = torch.device(device)

        def rows(h):
            return torch.empty((tokens, h * head_dim), dtype=self.dtype, device=dev)

        self.q_out, self.k_out = rows(n_q_heads), rows(n_k_heads)
        self.dq = self.dk = self.dgamma_q = self.dgamma_k = self.workspace = None
        if backward:
            self.dq, self.dk = rows(n_q_heads), rows(n_k_heads)
            self.dgamma_q = torch.empty((head_dim,), dtype=torch.float32, device=dev)
            self.dgamma_k = torch.empty((head_dim,), dtype=torch.float32, device=dev)
            ws = poetx_qk_norm_rope_backward_workspace_size(n_q_heads, n_k_heads, head_dim,
                                                            tokens, self.code)
            self.workspace = torch.empty((max(ws, 16),), dtype=torch.uint8, device=dev)

    def _ld(self, x, heads, t, name):
        """The row stride of one q / k tensor."""
        st = x.stride()
        if x.dtype is self.dtype and x.is_cuda and (
                (x.shape == (t, heads * self.D) and st[1] == 1) or
                (x.shape == (t, heads, self.D) and st[2] == 1 and st[1] == self.D)):
            return st[0]
        raise ValueError(f"{name}: rows of {heads * self.D} contiguous {self.dtype} elements for "
                         f"{t} tokens are needed, got {tuple(x.shape)}, {x.dtype}, strides {st}")

    def _check(self, gamma_q, gamma_k, cos, sin, positions, t):
        if t > self.tokens:
            raise ValueError(f"{t} tokens: the step holds buffers for {self.tokens}")
        for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
            if g is not None:
                _need(g, (self.D,), torch.float32, name)
        if self.rot:
            _need(cos, (cos.shape[0], self.rot // 2), torch.float32, "cos")
            _need(sin, (cos.shape[0], self.rot // 2), torch.float32, "sin")
        if positions is not None:
            _need(positions, (t,), torch.int32, "positions")
        return cos.shape[0] if self.rot else 0

    def _cut(self, buf, t):
        return buf if t == self.tokens else buf[:t]

    def forward(self, q, k, gamma_q, gamma_k, cos, sin, positions=None, stream=None):
        t = q.shape[0]
        rows = self._check(gamma_q, gamma_k, cos, sin, positions, t)
        ld_q = self._ld(q, self.hq, t, "q")
        ld_k = self._ld(k, self.hk, t, "k") if self.hk else 0
        poetx_qk_norm_rope_forward(q, k, gamma_q, gamma_k, cos, sin, positions, self.q_out,
                                   self.k_out, ld_q, ld_k, self.hq * self.D, self.hk * self.D,
                                   self.hq, self.hk, self.D, self.rot, rows, self.interleaved,
                                   self.eps, t, self.code, stream)
        return self._cut(self.q_out, t), self._cut(self.k_out, t)

    def backward(self, dq_out, dk_out, q, k, gamma_q, gamma_k, cos, sin, positions=None,
                 stream=None):
        """(dq, dk, dgamma_q, dgamma_k) from the outputs' gradients and the
        forward's inputs."""
        if self.dq is None:
            raise RuntimeError("PoetxQKNormRope was made without backward=True")
        t = q.shape[0]
        rows = self._check(gamma_q, gamma_k, cos, sin, positions, t)
        ld = [self._ld(dq_out, self.hq, t, "dq_out"),
              self._ld(dk_out, self.hk, t, "dk_out") if self.hk else 0,
              self._ld(q, self.hq, t, "q"), self._ld(k, self.hk, t, "k") if self.hk else 0]
        poetx_qk_norm_rope_backward(dq_out, dk_out, q, k, gamma_q, gamma_k, cos, sin, positions,
                                    self.dq, self.dk, self.dgamma_q, self.dgamma_k, *ld,
                                    self.hq * self.D, self.hk * self.D, self.hq, self.hk, self.D,
                                    self.rot, rows, self.interleaved, self.eps, t, self.code,
                                    self.workspace, stream)
        return self._cut(self.dq, t), self._cut(self.dk, t), self.dgamma_q, self.dgamma_k


def _need_list(tensors, others, dtypes, name):
    """Contiguous CUDA tensors of the types; `others` (or None) of the same sizes and types."""
    if not ({t.dtype for t in tensors} <= dtypes and
            all(map(torch.Tensor.is_contiguous, tensors)) and all(t.is_cuda for t in tensors)):
        raise ValueError(f"{name}: contiguous CUDA tensors of {sorted(map(str, dtypes))} are needed")
    if others is not None:
        _need_list(others, None, dtypes, "out")
        if [(t.numel(), t.dtype) for t in tensors] != [(t.numel(), t.dtype) for t in others]:
            raise ValueError(f"{name}: the lists differ in sizes or types")


class PoetxGradClip:
    """The global norm of a list of gradients (contiguous float32 or bfloat16
    tensors), and the clip to a largest norm.  self.norm is the norm of the
    last call (a 0-dim float32 tensor, overwritten by the next; undefined before the first)."""

    _TYPES = {torch.float32, torch.bfloat16}

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.norm = torch.empty((), dtype=torch.float32, device=self.device)
        self._spaces = []

    def _room(self, n):
        """A workspace for n tensors.  Smaller ones are kept: a call on another
        stream may still be using them."""
        need = poetx_grad_norm_workspace_size(n)
        if not self._spaces or self._spaces[-1].numel() < need:
            self._spaces.append(torch.empty((need,), dtype=torch.uint8, device=self.device))
        return self._spaces[-1]

    def total(self, grads, stream=None):
        """norm = sqrt(sum of squares over all tensors)."""
        _need_list(grads, None, self._TYPES, "grads")
        poetx_grad_norm(grads, self.norm, self._room(len(grads)), stream)
        return self.norm

    def clip(self, grads, max_norm, out=None, stream=None):
        """out (None: the gradients themselves) = grads * min(1, max_norm /
        (norm + 1e-6)); returns the norm before the clip."""
        _need_list(grads, out, self._TYPES, "grads")
        poetx_clip_grads(grads, out, max_norm, self.norm, self._room(len(grads)), stream)
        return self.norm
