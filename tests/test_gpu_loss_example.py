"""The example that uses the head's losses with a POET-X projection, the clip and Adam:
its gradients against the float64 oracles run one behind the other, and that it runs.

Bounds.  Relative Frobenius errors: a POET-X step in bf16 is within 2e-2 of its oracle
(the layer tests' bound), the losses' gradients within 2^-7 (loss_common: at most four
roundings of 2^-8 each, and these add in squares); hidden states off by 2^-8 move the
softmax's terms by their logits' change, 2^-8 of logits of a spread of 2 to 4: within
2e-2.  Together within 4e-2.  Scores: hidden states of the merged weight are 2^-8 apart
twice (weight and output), logits of up to 20 then by 20 * 2^-7 at most, and a loss by
twice that."""

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from oracle import loss_oracle as lo  # noqa: E402
from tests.block_common import host, status_ok  # noqa: E402

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "head_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    spec = importlib.util.spec_from_file_location("head_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def off(got, want):
    return np.linalg.norm(host(got).reshape(want.shape) - want) / np.linalg.norm(want)


def test_gradients(example):
    import orthogonal_reparameterized_packed_gb300 as px
    student, (x, targets, indices, logits) = example.start(seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in student.theta:
        t += torch.randn(t.shape, generator=g, device="cuda") * 0.02
    loss, grads = student.gradients(x, targets, indices, logits)
    status_ok(px)
    P, R = (host(t).astype(np.float32) for t in student.theta)
    W0, X, H = host(student.W0), host(x), host(student.head)
    b, k = example.BLOCK, example.ORDER
    zero = np.zeros_like(X)
    h = oracle.layer(P, R, W0, X, zero, b, k)["y"]
    ce = lo.cross_entropy(h, H, targets.cpu().numpy(), None)
    kd = lo.head_loss(h, H, indices.cpu().numpy(), host(logits), None, example.TEMPERATURE)
    want = oracle.layer(P, R, W0, X, ce[2] + example.SHARE * kd[2], b, k)
    assert abs(float(loss) - (ce[1] + example.SHARE * kd[1])) <= 2e-2 * ce[1]
    assert off(grads[0], want["dtheta_P"]) <= 4e-2
    assert off(grads[1], want["dtheta_R"]) <= 4e-2
    assert off(grads[2], ce[3] + example.SHARE * kd[3]) <= 4e-2


def test_it_runs(example):
    import orthogonal_reparameterized_packed_gb300 as px
    losses, apart = example.main(steps=5, quiet=True)
    assert px.poetx_device_status() == 0
    assert np.isfinite(losses).all() and apart <= 20 * 2.0 ** -6
