"""The losses at the output head where logits are not finite: an infinity in W that makes
a vocabulary entry impossible, one that makes it certain, and tokens that are not finite.
The bounds are those of loss_common, of the vocabulary without the impossible entry."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import loss_oracle as lo  # noqa: E402
from tests.block_common import EPS, host, status_ok, within  # noqa: E402
from tests.loss_common import bounds, check, device, make, rounded  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def head(c, tau, backward):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    kw = dict(dtype=c["dtype"], backward=backward, weight_grad=backward)
    if tau is None:
        return PoetxCrossEntropy(c["d"], c["V"], c["T"], **kw)
    return PoetxDistill(c["d"], c["V"], c["T"], top=c["K"], temperature=tau, **kw)


def one_more(T, d, V, tau, dtype):
    """A case of V entries, the same with one more, its number, and the feature at which its
    row of W is +inf: every token is negative there, so that its logits are -inf."""
    c = make(T, d, V, 1 if tau is None else 5, dtype, seed=T + V, ignored=0.1)
    j, at = d // 2, V // 3
    x = c["x"][1].copy()
    x[:, j] = -(np.abs(x[:, j]) + 0.5)
    c["x"] = rounded(x, dtype)
    W = np.insert(c["W"][1], at, c["W"][1][0], axis=0)
    W[at, j] = np.inf
    more = dict(c, V=V + 1, W=rounded(W, dtype), idx=c["idx"] + (c["idx"] >= at))
    return c, more, at, j


# rows behind the last up to a tile's end, and none; a weight whose products in fp32 run on
# the tensor cores where they are finite
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V", [(20, 64, 300), (70, 72, 500), (71, 128, 1000), (515, 512, 3001)])
def test_an_entry_of_minus_infinity(px, T, d, V, tau, dtype):
    """Its term is 0: losses and dW are those of the other entries, its own row of dW is 0;
    dx is NaN at W's infinity alone."""
    c, more, at, j = one_more(T, d, V, tau, dtype)
    want, bound = bounds(c, tau or 1.0, None, c["s"] if tau else np.zeros(c["idx"].shape))
    rest = device(more, tau is not None)
    h = head(more, tau, True)
    loss, dx, dW = h.step(more["x"][0], more["W"][0], *rest)
    status_ok(px)
    check((loss, h.total), want, bound)
    on = torch.from_numpy((c["idx"] >= 0).any(1)).cuda()
    assert dx[on, j].isnan().all() and not dx[~on].any()
    keep = np.arange(d) != j
    check((dx[:, torch.from_numpy(keep).cuda()],), (want[2][:, keep],), (bound[2][:, keep],),
          ("dx",))
    assert not dW[at].any()
    check((torch.cat((dW[:at], dW[at + 1:])),), want[3:], bound[3:], ("dW",))
    alone = head(more, tau, False)
    check((alone.forward(more["x"][0], more["W"][0], *rest), alone.total), want, bound)
    status_ok(px)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V", [(40, 64, 300), (90, 72, 500), (515, 512, 3001)])
def test_minus_infinity_at_an_own_entry(px, T, d, V, tau, dtype):
    """The token's loss is infinite, the other tokens keep their bits, and dW is the formula's:
    |dz| and |x| are rounded once each and dW's elements once (2^-8 or 2^-24), the softmax's
    terms are good to 2^-10: logits up to 32 off by d 2^-23 of themselves."""
    _, c, at, j = one_more(T, d, V, tau, dtype)
    h, alone = head(c, tau, True), head(c, tau, False)
    loss, dx, _ = (v.clone() for v in h.step(c["x"][0], c["W"][0], *device(c, tau is not None)))
    t = int(np.flatnonzero((c["idx"] >= 0).any(1))[3])
    c["idx"][t, 0] = at
    rest = device(c, tau is not None)
    got, gx, gw = h.step(c["x"][0], c["W"][0], *rest)
    status_ok(px)
    keep = torch.arange(T, device="cuda") != t
    on = torch.from_numpy((c["idx"] >= 0).any(1)).cuda()
    assert got[t] == float("inf") and h.total == float("inf")
    assert torch.equal(got[keep], loss[keep])
    assert torch.equal(gx[keep].nan_to_num(), dx[keep].nan_to_num())
    free = torch.arange(d, device="cuda") != j
    assert gx[on][:, free].isfinite().all() and not gx[on, j].isfinite().any()
    m = lo.head_loss(c["x"][1], c["W"][1], c["idx"], c["s"] if tau else np.zeros(c["idx"].shape),
                     None, tau or 1.0)
    dz, x = np.abs(m[4]["dz"]), np.abs(c["x"][1][m[4]["rows"]])
    q = m[4]["q"] * m[4]["w"][m[4]["rows"], None] * (tau or 1.0)
    u = EPS[dtype]
    within(host(gw), m[3], (3.1 * u * dz + 2.0 ** -10 * q + T * 2.0 ** -23 * dz).T @ x +
           u * np.abs(m[3]) + 2.0 ** -109 * T, "dW")
    got = alone.forward(c["x"][0], c["W"][0], *rest)
    assert got[t] == float("inf") and got[keep].isfinite().all()
    status_ok(px)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T", [40, 90])
def test_an_entry_of_infinity(px, T, tau, dtype):
    """In one token, at an entry that is none of its own: its loss is infinite, its dx and
    with it dW are NaN; the others keep their bits."""
    _, c, at, j = one_more(T, 64, 300, tau, dtype)
    rest = device(c, tau is not None)
    t = int(np.flatnonzero((c["idx"] >= 0).any(1))[3])
    x = c["x"][0].clone()
    x[t, j] = 1.0
    keep = torch.arange(T, device="cuda") != t
    h = head(c, tau, True)
    loss, dx, _ = (v.clone() for v in h.step(c["x"][0], c["W"][0], *rest))
    got, gx, gw = h.step(x, c["W"][0], *rest)
    status_ok(px)
    assert got[t] == float("inf") and h.total == float("inf")
    assert torch.equal(got[keep], loss[keep])
    assert torch.equal(gx[keep].nan_to_num(), dx[keep].nan_to_num())
    assert gx[t].isnan().all() and gw.isnan().all()
    alone = head(c, tau, False)
    loss = alone.forward(c["x"][0], c["W"][0], *rest).clone()
    got = alone.forward(x, c["W"][0], *rest)
    status_ok(px)
    assert got[t] == float("inf") and alone.total == float("inf")
    assert torch.equal(got[keep], loss[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T", [40, 90])
def test_tokens_that_are_not_finite(px, T, tau, dtype):
    """Losses and gradients of the others keep their bits; every row of dW is NaN."""
    c = make(T, 64, 300, 1 if tau is None else 5, dtype, seed=9)
    rest = device(c, tau is not None)
    x = c["x"][0].clone()
    x[3, 5], x[17, 0] = float("nan"), float("inf")
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[3] = keep[17] = False
    h = head(c, tau, True)
    loss, dx, _ = (v.clone() for v in h.step(c["x"][0], c["W"][0], *rest))
    got, gx, gw = h.step(x, c["W"][0], *rest)
    status_ok(px)
    assert torch.equal(got[keep], loss[keep]) and torch.equal(gx[keep], dx[keep])
    assert got[3].isnan() and not got[17].isfinite()
    assert gx[3].isnan().all() and not gx[17].isfinite().any() and gw.isnan().all()
    alone = head(c, tau, False)
    loss = alone.forward(c["x"][0], c["W"][0], *rest).clone()
    got = alone.forward(x, c["W"][0], *rest)
    status_ok(px)
    assert torch.equal(got[keep], loss[keep])
    assert got[3].isnan() and not got[17].isfinite() and not alone.total.isfinite()
