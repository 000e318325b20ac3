"""fp32 losses at the output head with weights of the tokens near the smallest that fp32
holds, where the products run on the CUDA cores: gradients scale with the weights."""

import pytest

torch = pytest.importorskip("torch")

from tests.block_common import status_ok  # noqa: E402
from tests.loss_common import device, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def gradients(px, T, d, V, tau):
    """dx and dW for weights, and for 2^-108 of them scaled back."""
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    c = make(T, d, V, 1 if tau is None else 5, "f32", seed=T, ignored=0.1)
    kw = dict(dtype="f32", backward=True, weight_grad=True)
    h = (PoetxCrossEntropy(d, V, T, **kw) if tau is None else
         PoetxDistill(d, V, T, top=5, temperature=tau, **kw))
    rest = device(c, tau is not None)
    w = torch.from_numpy(c["w"]).float().cuda()
    want = [v.double() for v in h.step(c["x"][0], c["W"][0], *rest, w)[1:]]
    got = h.step(c["x"][0], c["W"][0], *rest, w * 2.0 ** -108)[1:]
    status_ok(px)
    return [(g.double() * 2.0 ** 108, v) for g, v in zip(got, want)]


@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V", [(20, 64, 300), (130, 72, 100), (5, 100, 1000)])
def test_products_on_the_cuda_cores(px, T, d, V, tau):
    """2^-108 of a weight is exact, and so is everything that it multiplies but where a
    value comes below 2^-126: it is then off by 2^-150 at most, and weights are 2^-4 or more,
    their gradients' terms 2^-112 at the entries: 2^-38 of these, each of V or T times."""
    for got, want in gradients(px, T, d, V, tau):
        assert (got - want).norm() / want.norm() <= max(T, V) * 2.0 ** -37


@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V", [(700, 640, 3001), (333, 768, 8001)])
def test_products_on_the_tensor_cores(px, T, d, V, tau):
    """The small ones are left to the CUDA cores, whose sums are rounded otherwise: a sum
    of n terms of either sign is off by 2^-24 sqrt(n / 6) of its size in the mean, the six
    products of the other side by less than 2^-22."""
    for got, want in gradients(px, T, d, V, tau):
        assert (got - want).norm() / want.norm() <= 2.0 ** -24 * max(T, V) ** 0.5 + 2.0 ** -22
