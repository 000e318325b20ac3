"""The operators around the projections over their whole range: shapes drawn
with a fixed seed, sizes spread over their logarithm and odd ones among them,
compared with the float64 oracle by the parity tests' own bounds."""

import random

import pytest

torch = pytest.importorskip("torch")

from tests import test_gpu_linear as lin  # noqa: E402
from tests import test_gpu_optim as opt  # noqa: E402
from tests import test_gpu_qk_norm_rope as qk  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(24))
def test_linear(px, seed):
    rng = random.Random(1000 + seed)
    while True:
        T, a, b = log_int(rng, 1, 3000), log_int(rng, 1, 3000), log_int(rng, 1, 3000)
        if seed % 3:
            a, b = max(8, a - a % 8), max(8, b - b % 8)
        if T * a * b <= 4e8:
            break
    act, dtype = rng.choice(lin.ACTS), rng.choice(["bf16", "bf16", "f32"])
    lin.run_forward(px, T, a, b, dtype, act, rng.random() < .5, rng.random() < .5,
                    rng.random() < .5, seed)
    lin.run_backward(px, T, a, b, dtype, act, True, rng.random() < .5, seed)


@pytest.mark.parametrize("seed", range(32))
def test_qk_norm_rope(px, seed):
    rng = random.Random(2000 + seed)
    while True:
        T, hk = log_int(rng, 1, 4000), rng.choice([0, 1, 2, 3, 8, 12])
        hq = max(1, hk) * rng.choice([1, 2, 3, 8])
        D = rng.choice([16, 40, 48, 64, 72, 80, 96, 128, 160, 192, 256, log_int(rng, 1, 512)])
        if T * (hq + hk) * D <= 4e6:
            break
    rot = rng.choice([D, D // 2, rng.randint(0, D)])
    case = (T, hq, hk, D, rot - rot % 2, rng.random() < .5)
    dtype = rng.choice(["bf16", "f32"])
    pad, shift = rng.choice([0, 0, 8, 3]), rng.choice([0, 0, 4, 1])
    c = qk.Case(px, case, dtype, seed, pad=pad, shift=shift, gammas=rng.random() < .8)
    c.forward()
    qk.check_forward(c)
    c = qk.Case(px, case, dtype, seed, pad=pad, shift=shift, positions=rng.random() < .7)
    c.backward()
    qk.check_backward(c)


@pytest.mark.parametrize("seed", range(12))
def test_norm_clip_and_adam(px, seed, monkeypatch):
    rng = random.Random(3000 + seed)
    n = log_int(rng, 1, 600)
    most = max(2, 2000000 // n)
    monkeypatch.setattr(opt, "LISTS", [[rng.choice([0, 1, log_int(rng, 1, most)])
                                        for _ in range(n)]])
    dtypes = rng.choice([("f32",), ("bf16",), ("f32", "bf16"), ("bf16", "f32", "f32")])
    opt.test_norm_and_clip(px, 0, dtypes, rng.choice([0.5, 1e9]))
    opt.test_adam_matches_oracle(px, 0, rng.choice([None, 0.5, 1e9]))
