"""How far the losses at the output head and their gradients are off in the mean, against
float64 on the rounded inputs: what the worst-case bounds of loss_common leave open.

Logits.  The tensor core truncates its sum at every step of 16 of K: by half of 2^-23 of it
in the mean, and the sum grows as it goes, so a piece of k features loses k / 16 / 2 of
2^-24, k 2^-29 of itself.  Pieces are added up in registers, rounded to nearest.  A loss is
then off by that part of its logits, E_q |z| + |z_target|, at most; the rest (exponentials,
sums of the parts, the last operations) is below 2^-22 of them.  The mean square is held to
one and a half times k 2^-29, plus 2^-22: all of d = 4096 in one sum loses 7.6e-6.
bf16: pieces of 512, of 256 up to 256 rows, of 4096 / 16, 4096 / 8 and 4096 / 4 in the form
for few tokens (16, 8 and 4 sums).  fp32: pieces of 128, 2.4e-7, and half as much for the sum of the pieces;
operands with 16 of their 24 bits would leave 0.9e-6 to 1.3e-6 (evaluated in numpy).

Losses near 0 have their absolute error: the exponential of the target is good to 2^-22
(1.4e-7 in the mean), some ten additions round the sum of all to 2^-24 each (1e-7): 1.7e-7,
held to one and a half times that.  log2 of a sum 2^28 away in one number has 3.8e-7.

Gradients in bf16, in the norm: a rounding to bf16 leaves 1.66e-3 (of Gaussian values).
Cross entropy: dx has the result's, dW that and x times the factor's (2.35e-3); the error of
the entry's term is the factor's to take up, without which it were 2.35e-3 and 2.88e-3.
Distillation: one more each, which the factor takes up in part.
In fp32: products good to 2^-25, pieces of 128 truncated (2.4e-7), 2^-24 sqrt(n / 6) for the sum
of n pieces (up to 4e-7), the softmax's terms by their logits' errors, 3e-7 of up to 14, in a
part of the norm below 0.7: less than 2e-6 together.  Operands of 16 bits leave 9e-6."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import loss_oracle as lo  # noqa: E402
from tests.block_common import host, status_ok  # noqa: E402
from tests.loss_common import device, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def head(d, V, T, dtype, tau=None, top=1, backward=True, block=None):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    kw = dict(dtype=dtype, backward=backward, weight_grad=backward, block_tokens=block)
    if tau is None:
        return PoetxCrossEntropy(d, V, T, **kw)
    return PoetxDistill(d, V, T, top=top, temperature=tau, **kw)


def rms(a):
    return float(torch.as_tensor(a).double().square().mean().sqrt())


def logits_case(T, d, V, dtype):
    """x leans to an entry that is not its target: the loss is a difference of two logits."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    W = (torch.randn((V, d), generator=g, device="cuda") * (4.0 * d ** -0.5)).to(dt)
    at = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (torch.randn((T, d), generator=g, device="cuda") + 2.0 * W[at].float()).to(dt)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    z = x.double() @ W.double().t()
    lse = torch.logsumexp(z, 1, keepdim=True)
    of_target = z.gather(1, t[:, None])[:, 0]
    size = ((z - lse).exp() * z.abs()).sum(1) + of_target.abs()
    return x, W, t, lse[:, 0] - of_target, size


# the form that keeps terms and the one that does not, and the one for few tokens, whose
# weight fills the GPU with whole columns of K
@pytest.mark.parametrize("T,d,V,backward,piece", [
    (200, 1600, 1500, True, 256), (200, 1600, 1500, False, 256), (3, 2048, 1500, True, 256),
    (200, 4096, 1500, True, 256), (200, 4096, 1500, False, 256), (300, 1600, 1500, True, 512),
    (300, 2048, 1500, False, 512), (300, 4096, 1500, True, 512), (300, 4096, 1500, False, 512),
    (1, 4096, 32000, False, 256), (24, 4096, 32000, False, 512), (64, 4096, 32000, False, 1024)])
def test_losses_of_long_sums(px, T, d, V, backward, piece):
    x, W, t, want, size = logits_case(T, d, V, "bf16")
    h = head(d, V, T, "bf16", backward=backward)
    loss = h.step(x, W, t)[0] if backward else h.forward(x, W, t)
    status_ok(px)
    tol = 1.5 * piece * 2.0 ** -29 + 2.0 ** -22
    assert rms(loss.double() - want) <= tol * rms(size)
    assert abs(float(h.total) - float(want.mean())) <= tol * rms(size)


@pytest.mark.parametrize("T,d,V,backward", [
    (200, 4096, 1500, True), (515, 1000, 5000, True), (515, 1000, 5000, False),
    (300, 2048, 1100, True), (24, 512, 3000, False), (1, 2048, 5000, False)])
def test_losses_in_fp32(px, T, d, V, backward):
    x, W, t, want, size = logits_case(T, d, V, "f32")
    h = head(d, V, T, "f32", backward=backward)
    loss = h.step(x, W, t)[0] if backward else h.forward(x, W, t)
    status_ok(px)
    assert rms(loss.double() - want) <= 5e-7 * rms(size)
    assert abs(float(h.total) - float(want.mean())) <= 5e-7 * rms(size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,backward", [(300, True), (300, False), (40, True), (40, False)])
def test_losses_near_zero(px, T, backward, dtype):
    d, V = 256, 3001  # a short sum, whose error is none of these losses'
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    W = torch.randn((V, d), generator=g, device="cuda")
    W = (W / W.norm(dim=1, keepdim=True)).to(dt)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (torch.randn((T, d), generator=g, device="cuda") + 14.7 * W[t].float()).to(dt)
    z = x.double() @ W.double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0]
    assert 5e-4 < float(want.median()) < 5e-3
    h = head(d, V, T, dtype, backward=backward)
    loss = h.step(x, W, t)[0] if backward else h.forward(x, W, t)
    status_ok(px)
    # a change of the logits by d 2^-29 changes these losses by that part of themselves
    off = 1.5 * (1.7e-7 + d * 2.0 ** -29 * float(z.amax()) * rms(want))
    assert rms(loss.double() - want) <= off


def gradients(px, c, tau, block=None):
    """Errors of dx and dW in the norm."""
    h = head(c["d"], c["V"], c["T"], c["dtype"], tau, c["K"], block=block)
    _, dx, dW = h.step(c["x"][0], c["W"][0], *device(c, tau is not None))
    status_ok(px)
    logits = np.zeros(c["idx"].shape) if tau is None else c["s"]
    want = lo.head_loss(c["x"][1], c["W"][1], c["idx"], logits, None, tau or 1.0)[2:4]
    return [np.linalg.norm(host(g) - w) / np.linalg.norm(w) for g, w in zip((dx, dW), want)]


@pytest.mark.parametrize("T,d,V,block", [(130, 512, 1099, None), (513, 256, 1024, None),
                                         (300, 1024, 2000, 128), (64, 256, 3000, None)])
def test_gradients_of_cross_entropy_in_bf16(px, T, d, V, block):
    dx, dW = gradients(px, make(T, d, V, 1, "bf16", seed=T + d), None, block)
    assert dx <= 2.0e-3 and dW <= 2.6e-3


@pytest.mark.parametrize("T,d,V,K", [(260, 96, 3000, 64), (300, 512, 2000, 16)])
def test_gradients_of_distillation_in_bf16(px, T, d, V, K):
    dx, dW = gradients(px, make(T, d, V, K, "bf16", seed=T + d), 2.0)
    assert dx <= 2.4e-3 and dW <= 2.95e-3


# slices of dx, dW from kept planes, blocks whose last is ragged
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V,block", [(515, 1000, 5000, None), (300, 2048, 1100, None),
                                         (700, 640, 9001, 321), (333, 768, 8001, None),
                                         (64, 512, 9000, None), (40, 72, 600, None)])
def test_gradients_in_fp32(px, T, d, V, block, tau):
    c = make(T, d, V, 1 if tau is None else 7, "f32", seed=T + d, ignored=0.1)
    dx, dW = gradients(px, c, tau, block)
    assert dx <= 2e-6 and dW <= 2e-6
