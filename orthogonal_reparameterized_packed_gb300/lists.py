"""Lists of tensors as the C calls take them: host arrays of addresses, sizes and
types.  The calls read all their lists up to one count, so no list reaches them
that was not looked over here."""

from __future__ import annotations

import array

import torch

from . import BF16, F32

_EITHER = {torch.float32, torch.bfloat16}


def described(tensors, name, bf16=False):
    """(tensors, counts, types) of any iterable of contiguous CUDA tensors, float32 or,
    with bf16, bfloat16 too: the tensors as a list (a list itself) and the host array of
    their sizes."""
    if type(tensors) is not list:
        tensors = list(tensors)
    kinds = [t.dtype for t in tensors]
    if not ((kinds.count(torch.float32) == len(kinds) or bf16 and set(kinds) <= _EITHER) and
            all(map(torch.Tensor.is_contiguous, tensors)) and all([t.is_cuda for t in tensors])):
        raise ValueError(f"{name}: contiguous CUDA tensors of type float32"
                         f"{' or bfloat16' if bf16 else ''} are needed")
    return tensors, array.array("q", map(torch.Tensor.numel, tensors)), kinds


def same(name, got, want):
    """Raises unless the sizes (and types) of two lists that go together agree."""
    if got != want:
        raise ValueError(f"{name}: the lists differ in sizes or types")


def pointers(tensors):
    """(host array of the device pointers, its address); the array is to be kept alive."""
    a = array.array("Q", map(torch.Tensor.data_ptr, tensors))
    return a, a.buffer_info()[0]


def codes(kinds):
    """(host array of poetx_dtype, its address), or no array if all are float32."""
    if torch.bfloat16 not in kinds:
        return None, None
    a = array.array("i", [BF16 if k is torch.bfloat16 else F32 for k in kinds])
    return a, a.buffer_info()[0]
