"""A head outside the limits is refused when its object is made, before any buffer is (no
GPU needed)."""

import pytest
import torch

from orthogonal_reparameterized_packed_gb300.build import build_library
from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill


@pytest.fixture(autouse=True)
def no_buffers(monkeypatch):
    build_library()

    def empty(*a, **kw):
        raise AssertionError("a buffer was made")

    monkeypatch.setattr(torch, "empty", empty)


KW = dict(device="cpu", backward=True, weight_grad=True)


@pytest.mark.parametrize("temperature", [0.0, -1.0, 0.01, 64.5, 100, float("nan"), float("inf")])
def test_temperatures(temperature):
    with pytest.raises(ValueError, match="temperature"):
        PoetxDistill(64, 1000, 8, top=4, temperature=temperature, **KW)


@pytest.mark.parametrize("tokens", [0, 1, 8])
@pytest.mark.parametrize("d,vocab,top", [(0, 10, 1), (64, 0, 1), ((1 << 20) + 1, 10, 1),
                                         (64, (1 << 20) + 1, 1), (64, 10, 0), (64, 10, 1025)])
def test_sizes(tokens, d, vocab, top):
    with pytest.raises(ValueError, match="limits"):
        PoetxDistill(d, vocab, tokens, top=top, **KW)
    if top == 1:
        with pytest.raises(ValueError, match="limits"):
            PoetxCrossEntropy(d, vocab, tokens, **KW)


@pytest.mark.parametrize("tokens", [-1, (1 << 22) + 1])
def test_tokens(tokens):
    with pytest.raises(ValueError, match="limits"):
        PoetxCrossEntropy(64, 1000, tokens, **KW)
    with pytest.raises(ValueError, match="limits"):
        PoetxDistill(64, 1000, tokens, top=4, **KW)


def test_blocks():
    with pytest.raises(ValueError, match="limits"):
        PoetxCrossEntropy(64, 1000, 8, block_tokens=(1 << 22) + 1, **KW)


def test_what_is_inside(monkeypatch):
    made = []
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(a) or torch.zeros(1))
    for tokens in (0, 8):
        PoetxCrossEntropy(64, 1000, tokens, **KW)
        for t in (1 / 64, 1, 64):
            PoetxDistill(64, 1000, tokens, top=4, temperature=t, **KW)
    assert len(made) == 8 * 5
