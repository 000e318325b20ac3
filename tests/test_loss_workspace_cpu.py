"""What the workspace of the head's losses holds by form, as include/poetx.h states it (no
GPU needed)."""

import pytest

import orthogonal_reparameterized_packed_gb300 as poetx
from orthogonal_reparameterized_packed_gb300.build import build_library

B, F = poetx.BF16, poetx.F32
GIB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def library():
    build_library()


def size(d, V, T, code, gradients, block=0):
    return poetx.poetx_cross_entropy_workspace_size(d, V, T, code, gradients, block)


def rows(d, T, es):
    """The gathered x and what is kept per token (60 bytes), both rounded up."""
    return (T + 64) * (es * d + 64) + (64 << 10)


SIZES = [(4096, 128256, 4096), (2048, 32000, 8192), (2048, 32000, 65536), (1024, 1 << 20, 8192)]


def block_of(V, es, T):
    return min(2 * GIB // es // V, T + 64)


@pytest.mark.parametrize("d,V,T", SIZES)
def test_bf16_losses_keep_no_logit(d, V, T):
    terms = 2 * V * block_of(V, 2, T)
    assert size(d, V, T, B, 0) <= rows(d, T, 2) + terms // 16 + (1 << 20)


CUT = 160 << 20  # tiles of the products cut along K, dx' parts


@pytest.mark.parametrize("d,V,T", SIZES)
def test_bf16_gradients_keep_a_block_of_terms(d, V, T):
    terms = 2 * V * block_of(V, 2, T)
    one = rows(d, T, 2) + terms + terms // 16 + CUT + V * 128
    for gradients in (1, 2, 3):
        several = 4 * V * d if gradients & 2 and terms < 2 * V * T else 0
        assert size(d, V, T, B, gradients) <= one + several
    # smaller blocks: less for the terms, with dW its sums in fp32 besides
    assert size(d, V, T, B, 1, 1024) <= rows(d, T, 2) + 2 * V * 1024 * 17 // 16 + CUT + V * 2048
    assert 4 * V * d <= size(d, V, T, B, 3, 1024) - 2 * V * 1024 <= (
        rows(d, T, 2) + V * 128 + CUT + 4 * V * d + V * 2048)


@pytest.mark.parametrize("d,V,T", SIZES)
def test_f32_keeps_a_block_of_logits_and_their_planes(d, V, T):
    block = block_of(V, 4, T)
    logits = 4 * V * block
    split = (V + block + 128) * (6 * (d + 64) + 4 * (d // 1024 + 2))
    assert size(d, V, T, F, 0) <= rows(d, T, 4) + logits + split + (1 << 20)
    for gradients in (1, 2, 3):
        flags = 4 * block * (V // 1024 + 2)
        out = max(64 << 20, 4 * block * d)
        assert size(d, V, T, F, gradients) <= (rows(d, T, 4) + logits + logits * 3 // 2 +
                                               6 * 64 * block + 6 * 64 * V + flags + split + out +
                                               (1 << 20))


def test_blocks_can_take_more():
    """4096 tokens, 4096 -> 128256: 1.07 GiB whole, 2.51 in blocks of 2048 where the head is
    trained, 0.29 in blocks of 1024 where it is frozen."""
    at = (4096, 128256, 4096, B)
    assert size(*at, 3) < 1.1 * GIB < 2.4 * GIB < size(*at, 3, 2048)
    assert size(*at, 1, 1024) < 0.3 * GIB
