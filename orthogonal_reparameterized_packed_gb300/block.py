"""What stands around the projections in a decoder block: the matrix product
with bias, activation and residual (for frozen or merged weights), the norm of
queries and keys with the rotary embedding, and the clip of the gradients.
Each class holds the output buffers and the workspace of one such step and
enqueues its calls on a stream (the current one by default); calls of one object
on several streams have to be ordered by the caller (but for PoetxGradClip)."""

from __future__ import annotations

import torch

from . import (ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, _allocating_on, _check,
               _stream, load_library, poetx_grad_norm_workspace_size,
               poetx_linear_backward_workspace_size, poetx_linear_forward_workspace_size,
               poetx_qk_norm_rope_backward_workspace_size)
from .layer import _TORCH_DTYPE, dtype_code
from .lists import codes, described, pointers, same

# These classes call the library directly: a call for one token costs the host
# about as long as the GPU.

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU,
               "gelu_tanh": ACT_GELU_TANH}


def _need(t, shape, dtype, name):
    """The address of t, a contiguous CUDA tensor of this shape and type."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    raise ValueError(f"{name}: a contiguous CUDA tensor of shape {tuple(shape)} and type {dtype} "
                     f"is needed, got {tuple(t.shape)}, {t.dtype}, {t.device}")


def _address(t):
    return None if t is None else t.data_ptr()


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
        lib = load_library()
        self._fwd, self._bwd = lib.poetx_linear_forward, lib.poetx_linear_backward

    def _too_many(self, t):
        raise ValueError(f"{t} tokens: the layer holds buffers for {self.tokens}")

    def forward(self, x, W, bias=None, residual=None, stream=None):
        """y for x's tokens (a view of the layer's buffer; so is z, kept in
        self.z's first rows)."""
        t = x.shape[0]
        if t > self.tokens:
            self._too_many(t)
        _check("poetx_linear_forward", self._fwd(
            _need(x, (t, self.d_in), self.dtype, "x"),
            _need(W, (self.d_out, self.d_in), self.dtype, "W"),
            None if bias is None else _need(bias, (self.d_out,), torch.float32, "bias"),
            None if residual is None else _need(residual, (t, self.d_out), self.dtype, "residual"),
            self.y.data_ptr(), _address(self.z), self.d_in, self.d_out, t, self.act, self.code,
            self.workspace.data_ptr(), self.workspace.numel(), _stream(stream)))
        return self.y if t == self.tokens else self.y[:t]

    def backward(self, dy, W, z=None, stream=None):
        """(dx, dbias) from dy and the z of the forward (self.z by default);
        the residual's gradient is dy."""
        if self.dx is None:
            raise RuntimeError("PoetxLinear was made without backward=True")
        t = dy.shape[0]
        if t > self.tokens:
            self._too_many(t)
        z = self.z if z is None else z
        z_at = None
        if self.act != ACT_NONE:
            if z is None:
                raise ValueError("the backward of an activation needs z (save_z=True)")
            z_at = _need(z if z.shape[0] == t else z[:t], (t, self.d_out), self.dtype, "z")
        _check("poetx_linear_backward", self._bwd(
            _need(dy, (t, self.d_out), self.dtype, "dy"), z_at,
            _need(W, (self.d_out, self.d_in), self.dtype, "W"), self.dx.data_ptr(),
            self.dbias.data_ptr(), self.d_in, self.d_out, t, self.act, self.code,
            self.workspace.data_ptr(), self.workspace.numel(), _stream(stream)))
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
    fused projection).  cos, sin: [rows][rot_dim / 2] float32 (rope_tables);
    a token whose position is outside their rows gets zeros, no gradient, and sets the
    status word (poetx_device_status)."""

    def __init__(self, n_q_heads, n_k_heads, head_dim, tokens, rot_dim=None, eps=1e-6,
                 interleaved=False, dtype="bf16", device="cuda", backward=False):
        self.hq, self.hk, self.D, self.tokens = n_q_heads, n_k_heads, head_dim, tokens
        self.rot = head_dim if rot_dim is None else rot_dim
        self.eps, self.interleaved = eps, int(bool(interleaved))
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
            # without key heads no call writes it: the sum over no rows
            self.dgamma_k = (torch.empty if n_k_heads else torch.zeros)(
                (head_dim,), dtype=torch.float32, device=dev)
            ws = poetx_qk_norm_rope_backward_workspace_size(n_q_heads, n_k_heads, head_dim,
                                                            tokens, self.code)
            self.workspace = torch.empty((max(ws, 16),), dtype=torch.uint8, device=dev)
        lib = load_library()
        self._fwd = lib.poetx_qk_norm_rope_forward
        self._bwd = lib.poetx_qk_norm_rope_backward
        self._wq, self._wk = n_q_heads * head_dim, n_k_heads * head_dim

    def _rows(self, x, heads, t, name):
        """(address, row stride) of one q / k tensor."""
        st = x.stride()
        if x.dtype is self.dtype and x.is_cuda and (
                (x.shape == (t, heads * self.D) and st[1] == 1) or
                (x.shape == (t, heads, self.D) and st[2] == 1 and st[1] == self.D)):
            return x.data_ptr(), st[0]
        raise ValueError(f"{name}: rows of {heads * self.D} contiguous {self.dtype} elements for "
                         f"{t} tokens are needed, got {tuple(x.shape)}, {x.dtype}, strides {st}")

    def _small(self, gamma_q, gamma_k, cos, sin, positions, t):
        """Addresses of the weights, tables and positions, and the tables' rows."""
        if t > self.tokens:
            raise ValueError(f"{t} tokens: the step holds buffers for {self.tokens}")
        rows = cos.shape[0] if self.rot else 0
        trig = (rows, self.rot // 2)
        return (None if gamma_q is None else _need(gamma_q, (self.D,), torch.float32, "gamma_q"),
                None if gamma_k is None else _need(gamma_k, (self.D,), torch.float32, "gamma_k"),
                _need(cos, trig, torch.float32, "cos") if self.rot else None,
                _need(sin, trig, torch.float32, "sin") if self.rot else None,
                None if positions is None else _need(positions, (t,), torch.int32, "positions"),
                rows)

    def _cut(self, buf, t):
        return buf if t == self.tokens else buf[:t]

    def forward(self, q, k, gamma_q, gamma_k, cos, sin, positions=None, stream=None):
        t = q.shape[0]
        gq, gk, c, s, pos, rows = self._small(gamma_q, gamma_k, cos, sin, positions, t)
        q_at, ld_q = self._rows(q, self.hq, t, "q")
        k_at, ld_k = self._rows(k, self.hk, t, "k") if self.hk else (None, 0)
        _check("poetx_qk_norm_rope_forward", self._fwd(
            q_at, k_at, gq, gk, c, s, pos, self.q_out.data_ptr(), self.k_out.data_ptr(), ld_q,
            ld_k, self._wq, self._wk, self.hq, self.hk, self.D, self.rot, rows,
            self.interleaved, self.eps, t, self.code, _stream(stream)))
        return self._cut(self.q_out, t), self._cut(self.k_out, t)

    def backward(self, dq_out, dk_out, q, k, gamma_q, gamma_k, cos, sin, positions=None,
                 stream=None):
        """(dq, dk, dgamma_q, dgamma_k) from the outputs' gradients and the
        forward's inputs."""
        if self.dq is None:
            raise RuntimeError("PoetxQKNormRope was made without backward=True")
        t = q.shape[0]
        gq, gk, c, s, pos, rows = self._small(gamma_q, gamma_k, cos, sin, positions, t)
        dq_at, ld_dq = self._rows(dq_out, self.hq, t, "dq_out")
        q_at, ld_q = self._rows(q, self.hq, t, "q")
        dk_at = k_at = None
        ld_dk = ld_k = 0
        if self.hk:
            dk_at, ld_dk = self._rows(dk_out, self.hk, t, "dk_out")
            k_at, ld_k = self._rows(k, self.hk, t, "k")
        _check("poetx_qk_norm_rope_backward", self._bwd(
            dq_at, dk_at, q_at, k_at, gq, gk, c, s, pos, self.dq.data_ptr(), self.dk.data_ptr(),
            self.dgamma_q.data_ptr(), self.dgamma_k.data_ptr(), ld_dq, ld_dk, ld_q, ld_k,
            self._wq, self._wk, self.hq, self.hk, self.D, self.rot, rows, self.interleaved,
            self.eps, t, self.code, self.workspace.data_ptr(), self.workspace.numel(),
            _stream(stream)))
        return self._cut(self.dq, t), self._cut(self.dk, t), self.dgamma_q, self.dgamma_k


class PoetxGradClip:
    """The global norm of a list (any iterable) of gradients, contiguous float32
    or bfloat16 tensors, and the clip to a largest norm.  self.norm is the norm of the last
    call (a 0-dim float32 tensor; undefined before the first).

    Every stream has a norm, overwritten by the next call on it, and a workspace of its
    own, so that calls of one object on several streams may run at one time.  A captured
    graph holds those of the stream that it was captured on: graphs captured on one
    stream with one object are not to be replayed at one time."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.norm = torch.empty((), dtype=torch.float32, device=self.device)
        self._of_stream = {}  # handle -> (norm, workspaces, tensors that the last one takes)
        lib = load_library()
        self._total, self._clip = lib.poetx_grad_norm, lib.poetx_clip_grads

    def _buffers(self, n, stream):
        """(norm's address, address and bytes of a workspace for n tensors, handle) of the
        stream.  Smaller workspaces are kept: a captured graph may hold them."""
        handle = _stream(stream)
        norm, rooms, most = self._of_stream.get(handle, (None, [], -1))
        if n > most:
            need = poetx_grad_norm_workspace_size(n)
            with _allocating_on(stream, self.device):
                if not rooms or rooms[-1].numel() < need:
                    rooms.append(torch.empty((need,), dtype=torch.uint8, device=self.device))
                if norm is None:
                    norm = torch.empty((), dtype=torch.float32, device=self.device)
            self._of_stream[handle] = norm, rooms, n
        self.norm = norm
        return norm.data_ptr(), rooms[-1].data_ptr(), rooms[-1].numel(), handle

    def total(self, grads, stream=None):
        """norm = sqrt(sum of squares over all tensors)."""
        grads, counts, kinds = described(grads, "grads", bf16=True)
        (at, at_p), (types, types_p) = pointers(grads), codes(kinds)
        _check("poetx_grad_norm", self._total(
            len(counts), at_p, counts.buffer_info()[0], types_p,
            *self._buffers(len(counts), stream)))
        return self.norm

    def clip(self, grads, max_norm, out=None, stream=None):
        """out (None: the gradients themselves) = grads * min(1, max_norm /
        (norm + 1e-6)); returns the norm before the clip."""
        grads, counts, kinds = described(grads, "grads", bf16=True)
        (at, at_p), (types, types_p) = pointers(grads), codes(kinds)
        to, to_p = at, at_p
        if out is not None:
            out, *like = described(out, "out", bf16=True)
            same("out", like, [counts, kinds])
            to, to_p = pointers(out)
        _check("poetx_clip_grads", self._clip(
            len(counts), at_p, to_p, counts.buffer_info()[0], types_p, max_norm,
            *self._buffers(len(counts), stream)))
        return self.norm
