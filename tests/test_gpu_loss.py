"""GPU parity of the losses at the output head and of their gradients, against the
float64 oracle on the rounded inputs.  The bounds are derived in loss_common."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.block_common import Guarded, host, status_ok  # noqa: E402
from tests.loss_common import bounds, check, device, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def head(c, tau, **kw):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    kw = {"backward": True, "weight_grad": True, "dtype": c["dtype"], **kw}
    tokens = kw.pop("tokens", c["T"])
    if tau is None:
        return PoetxCrossEntropy(c["d"], c["V"], tokens, **kw)
    return PoetxDistill(c["d"], c["V"], tokens, top=c["K"], temperature=tau, **kw)


def expected(c, tau, weights=None):
    if tau is None:
        return bounds(c, 1.0, weights, np.zeros((c["T"], c["K"])))
    return bounds(c, tau, weights, c["s"])


def run_and_check(px, c, tau, weights=None, **kw):
    h = head(c, tau, **kw)
    rest = device(c, tau is not None)
    w = None if weights is None else torch.from_numpy(weights).float().cuda()
    want, bound = expected(c, tau, weights)
    loss, dx, dW = h.step(c["x"][0], c["W"][0], *rest, w)
    status_ok(px)
    check((loss, h.total, dx, dW), want, bound)
    alone = h.forward(c["x"][0], c["W"][0], *rest, w)
    status_ok(px)
    check((alone, h.total), want, bound)
    return h


# (T, d, V): one token to several tiles and blocks of tiles, either side of the 64-,
# 128- and 256-wide tiles, odd ones, single elements
SHAPES = [(1, 1, 1), (1, 64, 128), (1, 512, 3001), (2, 8, 5), (3, 7, 300), (16, 256, 1000),
          (17, 72, 257), (24, 264, 2049), (33, 96, 255), (64, 128, 512), (65, 320, 777),
          (127, 40, 1030), (128, 64, 128), (130, 512, 4099), (255, 136, 640), (257, 192, 1281),
          (300, 1000, 513), (513, 256, 1024), (600, 65, 901), (2047, 64, 130), (2049, 72, 100), (1100, 128, 300), (70, 2048, 3000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_cross_entropy(px, T, d, V, dtype):
    c = make(T, d, V, 1, dtype, seed=T + d, ignored=0.2 if T > 2 else 0.0)
    run_and_check(px, c, None, c["w"] if V % 2 else None)


# either side of the pieces of K that the logits are summed in (768), several tiles of
# logits for a cluster of CTAs
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", [(70, 768, 300), (70, 776, 300), (130, 1600, 700),
                                   (90, 4096, 520), (600, 64, 9000), (64, 4096, 260),
                                   (20, 1536, 140)])
def test_long_and_wide(px, T, d, V, dtype):
    c = make(T, d, V, 1, dtype, seed=T + d, ignored=0.1)
    run_and_check(px, c, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,K,tau", [
    (1, 64, 300, 16, 2.0), (1, 9, 4, 3, 1.0), (5, 128, 1000, 1, 1.0), (40, 256, 2051, 7, 4.0),
    (129, 192, 515, 33, 0.5), (260, 96, 3000, 64, 1.5), (33, 72, 100, 100, 3.0),
    (300, 320, 1300, 20, 1.0), (12, 64, 5000, 1024, 2.0), (515, 512, 777, 130, 64.0),
    (2048, 72, 130, 3, 2.0), (2049, 64, 300, 5, 2.0)])
def test_distill(px, T, d, V, K, tau, dtype):
    c = make(T, d, V, K, dtype, seed=T + K, ignored=0.3 if T > 2 else 0.0)
    run_and_check(px, c, tau, c["w"] if T % 2 else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("block", [1, 64, 100, 256])
def test_blocks_of_tokens(px, tau, dtype, block):
    c = make(300, 136, 700, 1 if tau is None else 9, dtype, seed=block, ignored=0.25)
    run_and_check(px, c, tau, block_tokens=block)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 1.0])
@pytest.mark.parametrize("x_scale", [0.0, 30.0, 400.0])
def test_logits_of_any_size(px, tau, dtype, x_scale):
    """All equal; hundreds apart; thousands apart, with targets far below the largest."""
    c = make(140, 64, 900, 1 if tau is None else 5, dtype, seed=3, x_scale=x_scale)
    rng = np.random.default_rng(4)
    c["idx"] = rng.integers(0, 900, c["idx"].shape)  # not the ones that x leans to
    run_and_check(px, c, tau)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
def test_some_blocks_with_wide_logits(px, tau, dtype):
    """Targets hundreds below the largest logit in some blocks of tokens only."""
    c = make(300, 72, 900, 1 if tau is None else 5, dtype, seed=11, ignored=0.1)
    c["idx"][100:130] = np.random.default_rng(5).integers(0, 900, c["idx"][100:130].shape)
    x = c["x"][0].clone()
    x[100:130] *= 64.0  # exact
    c["x"] = (x, host(x))
    for block in (None, 64):
        run_and_check(px, c, tau, c["w"], block_tokens=block)
    few = dict(c, T=20, idx=c["idx"][100:120], s=c["s"][100:120], w=c["w"][100:120],
               x=(x[100:120].clone(), host(x[100:120])))
    want, bound = expected(few, tau)
    h = head(few, tau, backward=False, weight_grad=False)
    loss = h.forward(few["x"][0], few["W"][0], *device(few, tau is not None))
    status_ok(px)
    check((loss, h.total), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,few", [(20, 1024, 1), (20, 130, 3), (150, 64, 5), (2100, 33, 2)])
def test_few_indices_many_times(px, T, K, few, dtype):
    """Every entry of a token at one of a few indices, some absent; their weights add up."""
    c = make(T, 64, 300, K, dtype, seed=K, ignored=0.1)
    rng = np.random.default_rng(K)
    own = rng.integers(0, 300, (T, few))
    at = np.take_along_axis(own, rng.integers(0, few, (T, K)), 1)
    at[:, 1:][rng.random((T, K - 1)) < 0.2] = -1
    at[(c["idx"] < 0).all(1)] = -1
    c["idx"] = at
    run_and_check(px, c, 2.0)


@pytest.mark.parametrize("T,d,V", [(300, 1100, 2048), (300, 2048, 1100), (300, 1500, 2048),
                                   (300, 3001, 1100), (200, 2048, 2048), (515, 1000, 5000)])
def test_f32_tile_widths_of_dw(px, T, d, V):
    c = make(T, d, V, 1, "f32", seed=d, ignored=0.1)
    run_and_check(px, c, None, c["w"])


@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V,block,tiny", [
    (515, 512, 5003, None, False), (700, 640, 9001, 321, False), (700, 640, 9001, 321, True)])
def test_f32_dw_alone_and_over_blocks(px, T, d, V, block, tiny, tau):
    """dW from planes that no dx product has made, and over blocks whose last is ragged;
    a value below 2^-109 in one block of tokens leaves that block to the CUDA cores."""
    c = make(T, d, V, 1 if tau is None else 5, "f32", seed=V + T, ignored=0.1)
    if tiny:
        t = c["x"][0].clone()
        t[T // 2, :7] = 1e-36
        c["x"] = (t, host(t))
    h = run_and_check(px, c, tau, block_tokens=block)
    want, bound = expected(c, tau)
    dW = h.dW.clone()
    h.dW.fill_(float("nan"))
    idx, *rest = device(c, tau is not None)
    out = (h.loss, h.total, None, h.dW, d, V, T)
    end = (px.F32, h.block_tokens, h.workspace)
    if tau is None:
        px.poetx_cross_entropy(c["x"][0], c["W"][0], idx, 8, None, *out, *end)
    else:
        px.poetx_distill(c["x"][0], c["W"][0], idx, 8, rest[0], px.F32, None, *out, c["K"], tau,
                         *end)
    status_ok(px)
    check((h.loss, h.total), want, bound)
    assert torch.equal(h.dW, dW)


@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V,block", [(64, 512, 9000, None), (300, 256, 5000, 128),
                                         (333, 768, 4001, None)])
def test_f32_values_that_the_tensor_cores_do_not_take(px, T, d, V, block, tau):
    """Below 2^-109, in a token and in W: their products on the CUDA cores, dx' slices too."""
    for where in ("x", "W"):
        c = make(T, d, V, 1 if tau is None else 5, "f32", seed=T, ignored=0.1)
        t = c[where][0].clone()
        t[3, :7] = 1e-36
        c[where] = (t, host(t))
        run_and_check(px, c, tau, block_tokens=block)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
def test_tokens_that_do_not_count(px, tau, dtype):
    """Their x, weights and logits may hold anything; rows behind the call's tokens keep
    what they hold."""
    c = make(150, 72, 500, 1 if tau is None else 6, dtype, seed=8, ignored=0.4)
    off = np.flatnonzero(c["idx"][:, 0] < 0)
    want, bound = expected(c, tau, c["w"])
    x, rest = c["x"][0].clone(), device(c, tau is not None)
    w = torch.from_numpy(c["w"]).float().cuda()
    at = torch.from_numpy(off).cuda()
    x[at[0::3]], x[at[1::3]], x[at[2::3]] = float("nan"), float("inf"), 3e38
    w[at] = float("nan")
    if tau is not None:
        rest[1][at] = float("nan")
    h = head(c, tau, tokens=200)
    h.loss.fill_(7.0)
    h.dx.fill_(7.0)
    loss, dx, dW = h.step(x, c["W"][0], *rest, w)
    status_ok(px)
    check((loss, h.total, dx, dW), want, bound)
    assert not loss[at].any() and not dx[at].any()
    assert (h.loss[150:] == 7).all() and (h.dx[150:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
def test_no_token_counts(px, tau, dtype):
    c = make(70, 64, 300, 1 if tau is None else 4, dtype, seed=1, ignored=1.0)
    c["x"][0].fill_(float("nan"))
    h = head(c, tau)
    for b in (h.loss, h.total, h.dx, h.dW):
        b.fill_(float("nan"))
    out = (*h.step(c["x"][0], c["W"][0], *device(c, tau is not None)), h.total)
    status_ok(px)
    assert all(not t.any() for t in out)
    assert not h.forward(c["x"][0], c["W"][0], *device(c, tau is not None)).any()


@pytest.mark.parametrize("tau", [None, 2.0])
def test_no_tokens(px, tau):
    c = make(8, 64, 300, 1 if tau is None else 4, "bf16", seed=1)
    h = head(c, tau)
    for b in (h.total, h.dW):
        b.fill_(float("nan"))
    loss, dx, dW = h.step(c["x"][0][:0], c["W"][0], *[a[:0] for a in device(c, tau is not None)])
    status_ok(px)
    assert loss.shape == (0,) and dx.shape == (0, 64) and h.total == 0 and not dW.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entries_of_every_kind(px, dtype):
    """Absent ones, the same index twice, -inf, the type's lowest value, NaN where no
    entry is; indices outside are not followed and set the status word."""
    c = make(12, 64, 90, 5, dtype, seed=5)
    idx, s = c["idx"], c["s"]
    idx[0] = [3, 3, 3, 8, 8]
    idx[1] = [-1, -7, 4, -100, 5]
    s[1] = [np.nan, np.inf, 1.0, 3e38, 2.0]
    s[2] = [1.0, -np.inf, 0.5, -np.inf, -np.inf]
    s[3] = -np.inf
    low = float(torch.finfo(torch.float32).min)
    s[4] = low
    s[5] = [0.0, low, low, 1.0, low]
    idx[6] = [89, 0, 89, 0, 1]
    s[7] = [-200.0, -100.0, 0.0, 80.0, 100.0]
    for tau in (0.25, 1.0, 8.0):
        run_and_check(px, c, tau)
    want, bound = expected(c, 1.0)
    outside = c["idx"].copy()
    outside[8] = [90, 1 << 20, 0, 0, 1]
    c["idx"] = outside
    want, bound = expected(c, 1.0)
    h = head(c, 1.0)
    idx64 = torch.from_numpy(outside).cuda()
    idx64[8, 1] = 1 << 40
    loss, dx, dW = h.step(c["x"][0], c["W"][0], idx64, torch.from_numpy(s).float().cuda())
    torch.cuda.synchronize()
    assert px.poetx_device_status() == 1 and px.poetx_device_status() == 0
    check((loss, h.total, dx, dW), want, bound)


def test_targets_outside(px):
    c = make(20, 64, 90, 1, "bf16", seed=6)
    c["idx"][3], c["idx"][4] = 90, -1
    want, bound = expected(c, None)
    h = head(c, None)
    t = device(c, False)[0]
    t[3] = 1 << 40
    loss, dx, dW = h.step(c["x"][0], c["W"][0], t)
    torch.cuda.synchronize()
    assert px.poetx_device_status() == 1 and px.poetx_device_status() == 0
    check((loss, h.total, dx, dW), want, bound)


@pytest.mark.parametrize("tau", [None, 2.0])
def test_types_of_indices_and_logits(px, tau):
    c = make(50, 64, 300, 1 if tau is None else 6, "bf16", seed=2, ignored=0.2)
    c["s"] = torch.from_numpy(c["s"]).bfloat16().double().numpy()
    h = head(c, tau)
    want, bound = expected(c, tau)
    for it in (torch.int32, torch.int64):
        for lt in (torch.float32, torch.bfloat16):
            rest = device(c, tau is not None, it)
            rest = (rest[0], *[r.to(lt) for r in rest[1:]])
            loss, dx, dW = h.step(c["x"][0], c["W"][0], *rest)
            status_ok(px)
            check((loss, h.total, dx, dW), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_that_are_not_finite(px, dtype):
    """A NaN or an infinite logit stays with its token: loss and dx of the others keep
    their bits."""
    c = make(40, 64, 300, 1, dtype, seed=9)
    h = head(c, None)
    t = device(c, False)[0]
    loss, dx, _ = h.step(c["x"][0], c["W"][0], t)
    loss, dx = loss.clone(), dx.clone()
    x = c["x"][0].clone()
    x[3, 5], x[17, 0] = float("nan"), float("inf")
    got, gx, gw = h.step(x, c["W"][0], t)
    status_ok(px)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[17] = False
    assert torch.equal(got[keep], loss[keep]) and torch.equal(gx[keep], dx[keep])
    assert got[3].isnan() and not got[17].isfinite()
    assert gx[3].isnan().all() and not gx[17].isfinite().any()
    assert gw.isnan().all(1).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V,block", [(1, 64, 300, 0), (37, 72, 513, 0), (300, 65, 257, 100),
                                         (130, 256, 1000, 0)])
def test_nothing_else_is_written(px, T, d, V, block, tau, dtype):
    """Outputs and a workspace of the stated size between guard bands."""
    K = 1 if tau is None else 5
    c = make(T, d, V, K, dtype, seed=T)
    code = px.BF16 if dtype == "bf16" else px.F32
    tdt = c["x"][0].dtype
    want, bound = expected(c, tau)
    for grads in (0, px.GRAD_X, px.GRAD_W, px.GRAD_X | px.GRAD_W):
        g = Guarded()
        loss, total = g.tensor((T,), torch.float32), g.tensor((1,), torch.float32)
        dx = g.tensor((T, d), tdt) if grads & px.GRAD_X else None
        dW = g.tensor((V, d), tdt) if grads & px.GRAD_W else None
        rest = device(c, tau is not None)
        if tau is None:
            ws = g.tensor((px.poetx_cross_entropy_workspace_size(d, V, T, code, grads, block),),
                          torch.uint8)
            px.poetx_cross_entropy(c["x"][0], c["W"][0], rest[0], 8, None, loss, total, dx, dW, d,
                                   V, T, code, block, ws)
        else:
            ws = g.tensor((px.poetx_distill_workspace_size(d, V, T, K, code, grads, block),),
                          torch.uint8)
            px.poetx_distill(c["x"][0], c["W"][0], rest[0], 8, rest[1], px.F32, None, loss, total,
                             dx, dW, d, V, T, K, tau, code, block, ws)
        g.check()
        status_ok(px)
        check((loss, total[0]), want, bound)
        if dx is not None:
            check((dx,), want[2:], bound[2:], ("dx",))
        if dW is not None:
            check((dW,), want[3:], bound[3:], ("dW",))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [None, 2.0])
def test_fewer_tokens_and_other_streams(px, tau, dtype):
    """One object for 1 to its tokens, on a stream of its own, twice the same bits; an object
    made for just that many."""
    K = 1 if tau is None else 5
    h = head(make(600, 128, 500, K, dtype, seed=0), tau)
    side = torch.cuda.Stream()
    for T in (600, 1, 65, 256, 257, 590):
        c = make(T, 128, 500, K, dtype, seed=T, ignored=0.1)
        rest = device(c, tau is not None)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            first = [v.clone() for v in (*h.step(c["x"][0], c["W"][0], *rest), h.total)]
        again = (*h.step(c["x"][0], c["W"][0], *rest, stream=side), h.total)
        side.synchronize()
        again = [v.clone() for v in again]
        own = head(c, tau)
        other = (*own.step(c["x"][0], c["W"][0], *rest), own.total)
        status_ok(px)
        want, bound = expected(c, tau)
        check((first[0], first[3], first[1], first[2]), want, bound)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        check((other[0], other[3], other[1], other[2]), want, bound)


@pytest.mark.parametrize("tau", [None, 2.0])
def test_captured_and_replayed(px, tau):
    """A captured step follows its inputs: other values, other counts of tokens that
    count, a wide row that takes another way through the kernels."""
    K = 1 if tau is None else 5
    c = make(200, 128, 700, K, "bf16", seed=0)
    h = head(c, tau)
    x, W, rest = c["x"][0].clone(), c["W"][0].clone(), device(c, tau is not None)
    h.step(x, W, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.step(x, W, *rest)
    for seed, ignored, scale in ((1, 0.0, 1.0), (2, 0.5, 1.0), (3, 0.0, 200.0), (4, 1.0, 1.0),
                                 (5, 0.1, 1.0)):
        n = make(200, 128, 700, K, "bf16", seed=seed, ignored=ignored, x_scale=scale)
        if scale > 1:
            n["idx"] = np.random.default_rng(seed).integers(0, 700, n["idx"].shape)
        x.copy_(n["x"][0])
        W.copy_(n["W"][0])
        for a, b in zip(rest, device(n, tau is not None)):
            a.copy_(b)
        graph.replay()
        status_ok(px)
        want, bound = expected(n, tau)
        check((h.loss, h.total, h.dx, h.dW), want, bound)


@pytest.mark.parametrize("tau", [None, 2.0])
def test_gradients_are_the_differences(px, tau):
    """fp32: total along a direction v of x (and of W), against <gradient, v>.  A central
    difference of step h is off by h^2 / 6 times the third derivative (a third cumulant of
    the logits' change, each at most 10 here: below 1000, times tau^2 / tau^3) and by the
    totals' errors over h."""
    c = make(30, 64, 200, 1 if tau is None else 5, "f32", seed=7, ignored=0.2)
    h = head(c, tau)
    rest = device(c, tau is not None)
    _, bound = expected(c, tau)
    _, dx, dW = h.step(c["x"][0], c["W"][0], *rest)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, grad in ((0, dx.clone()), (1, dW.clone())):
        a = (c["x"][0], c["W"][0])[i]
        v = torch.randn(a.shape, generator=g, device="cuda") / a.shape[1] ** 0.5
        step, totals = 2.0 ** -6, []
        for sign in (1, -1):
            moved = a + sign * step * v
            h.forward(*((moved, c["W"][0]) if i == 0 else (c["x"][0], moved)), *rest)
            totals.append(float(h.total))
        slope = (totals[0] - totals[1]) / (2 * step)
        want = float((grad.double() * v.double()).sum())
        # a + step v is rounded to 2^-24 of a's values (up to 16): its own change of total
        off = 2.0 ** -20 * float((grad.double().abs()).sum()) / step
        assert abs(slope - want) <= step ** 2 / 6 * 1000 + 2 * bound[1] / step + off


def test_long_rows_pass_32_bits(px):
    """Terms and gradients whose offsets pass 2^31 elements (bytes: 2^32), against the
    same head in blocks of tokens."""
    T, d, V = 4352, 64, 500009
    g = torch.Generator(device="cuda").manual_seed(0)
    W = (torch.randn((V, d), generator=g, device="cuda") * 0.25).bfloat16()
    x = torch.randn((T, d), generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy
    h = PoetxCrossEntropy(d, V, T, backward=True, weight_grad=True, block_tokens=T)
    loss, dx, dW = h.step(x, W, t)
    status_ok(px)
    rows = torch.tensor([0, 1, 255, 256, 4096, T - 1], device="cuda")
    z = x[rows].double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    want = lse - z[torch.arange(len(rows), device="cuda"), t[rows]]
    assert float((loss[rows].double() - want).abs().max()) <= 64 * 2.0 ** -23 * 64 + 1e-4
    q = (z - lse[:, None]).exp()
    q[torch.arange(len(rows), device="cuda"), t[rows]] -= 1
    gx = q @ W.double() / T
    scale = (q.abs() @ W.double().abs()) / T
    assert bool(((dx[rows].double() - gx).abs() <= 2.0 ** -6 * scale).all())
    del z, q
    few = PoetxCrossEntropy(d, V, T, backward=True, weight_grad=True, block_tokens=1024)
    loss2, dx2, dW2 = few.step(x, W, t)
    status_ok(px)
    assert float((loss2 - loss).abs().max()) <= 1e-4
    assert float((dx2.float() - dx.float()).abs().max()) <= 2.0 ** -6 * float(scale.max())
    off = float((dW2.float() - dW.float()).norm() / dW.float().norm())
    assert off <= 2 * 2.0 ** -7  # both rounded: terms, factors and results


@pytest.mark.parametrize("T,d,V", [(5000, 1024, 4000), (4200, 256, 20500), (6000, 1024, 300),
                                   (40, 1024, 30000), (8200, 64, 600)])
def test_rounds_of_tiles(px, T, d, V):
    """More tiles of dx or dW than clusters of CTAs, last rounds cut along K, few tiles of a
    long K.  The bounds of loss_common, evaluated in float64 on the GPU."""
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy
    g = torch.Generator(device="cuda").manual_seed(T)
    W = (torch.randn((V, d), generator=g, device="cuda") * 2 * d ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (torch.randn((T, d), generator=g, device="cuda") + 2.0 * W[t].float()).bfloat16()
    t[::7] = -1
    h = PoetxCrossEntropy(d, V, T, backward=True, weight_grad=True)
    loss, dx, dW = h.step(x, W, t)
    status_ok(px)
    on = t >= 0
    X, Y, H = x[on].double(), t[on], W.double()
    n, u = len(Y), 2.0 ** -8
    z = X @ H.t()
    rows = torch.arange(n, device="cuda")
    lse = torch.logsumexp(z, 1, keepdim=True)
    want = lse[:, 0] - z[rows, Y]
    ez = d * 2.0 ** -23 * float((X.abs() @ H.abs().t()).max())
    e_q = 2.1 * (ez + 2.0 ** -21 * (float(z.abs().max()) + 64) + 2.0 ** -21) + (
        512 + V / 128) * 2.0 ** -24
    assert bool(((loss[on].double() - want).abs() <= 2 * e_q + 2.0 ** -20 * (1 + want)).all())
    assert not loss[~on].any() and not dx[~on].any()
    q = (z - lse).exp()
    del z
    b = q * e_q / n
    q[rows, Y] -= 1
    dz = q / n
    del q
    top = 2.0 ** -20 / n
    for got, exact, size in (
            (dx[on].double(), dz @ H, (2 * u + V * 2.0 ** -23) * 1.02 * (dz.abs() @ H.abs()) +
             b @ H.abs() + top),
            (dW.double(), dz.t() @ X, (3 * u + T * 2.0 ** -23) * 1.03 * (dz.abs().t() @ X.abs()) +
             b.t() @ X.abs() + top * float(X.abs().max()))):
        size = size + u * (exact.abs() + size)
        assert bool(((got - exact).abs() <= size).all())


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T", [1, 5, 20, 64])
def test_scores_of_few_tokens(px, T, tau, index):
    """Losses alone of up to 64 tokens, with tokens that do not count and hold anything, and an
    index outside the vocabulary."""
    c = make(T, 128, 700, 1 if tau is None else 6, "bf16", seed=T)
    rng = np.random.default_rng(T)
    off = np.flatnonzero(rng.random(T) < 0.3) if T > 1 else np.zeros(0, dtype=int)
    c["idx"][off] = -5
    outside = T > 5
    if outside:
        c["idx"][2] = 700
    for weights in (None, c["w"]):
        want, bound = expected(c, tau, weights)
        x, rest = c["x"][0].clone(), device(c, tau is not None, index)
        x[torch.from_numpy(off).cuda()] = float("nan")
        w = None if weights is None else torch.from_numpy(weights).float().cuda()
        if w is not None:
            w[torch.from_numpy(off).cuda()] = float("inf")
        h = head(c, tau, backward=False, weight_grad=False)
        h.loss.fill_(9.0)
        loss = h.forward(x, c["W"][0], *rest, w)
        torch.cuda.synchronize()
        assert px.poetx_device_status() == (1 if outside else 0)
        check((loss, h.total), want, bound)
    if T > 1:  # none counts
        none = [torch.full_like(rest[0], -1), *rest[1:]]
        assert not h.forward(x, c["W"][0], *none).any() and h.total == 0


@pytest.mark.parametrize("tau", [None, 2.0])
def test_scores_captured(px, tau):
    K = 1 if tau is None else 6
    c = make(10, 128, 700, K, "bf16", seed=0)
    h = head(c, tau, backward=False, weight_grad=False)
    x, W, rest = c["x"][0].clone(), c["W"][0], device(c, tau is not None)
    h.forward(x, W, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.forward(x, W, *rest)
        h.forward(x, W, *rest)
    for seed in (1, 2):
        n = make(10, 128, 700, K, "bf16", seed=seed, ignored=0.3)
        x.copy_(n["x"][0])
        W.copy_(n["W"][0])
        for a, b in zip(rest, device(n, tau is not None)):
            a.copy_(b)
        graph.replay()
        status_ok(px)
        want, bound = expected(n, tau)
        check((h.loss, h.total), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_objects_at_once(px, dtype):
    """Two heads on two streams, enqueued in turn: both as alone."""
    cases = [make(300, 256, 2000, 1, dtype, seed=1), make(200, 512, 3000, 5, dtype, seed=2)]
    taus = [None, 2.0]
    heads = [head(c, t) for c, t in zip(cases, taus)]
    rest = [device(c, t is not None) for c, t in zip(cases, taus)]
    alone = []
    for h, c, r in zip(heads, cases, rest):
        out = (*h.step(c["x"][0], c["W"][0], *r), h.total)
        torch.cuda.synchronize()
        alone.append([v.clone() for v in out])
    streams = [torch.cuda.Stream() for _ in heads]
    torch.cuda.synchronize()
    for _ in range(5):
        for h, c, r, s in zip(heads, cases, rest, streams):
            h.step(c["x"][0], c["W"][0], *r, stream=s)
    torch.cuda.synchronize()
    status_ok(px)
    for h, want in zip(heads, alone):
        assert all(torch.equal(a, b) for a, b in zip((h.loss, h.dx, h.dW, h.total), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_every_size(px, dtype):
    """Weights 2^60 apart, negative ones and zeros: each token's gradient has its own."""
    c = make(90, 64, 400, 1, dtype, seed=4)
    c["w"] = c["w"] * np.where(np.arange(90) % 3 == 0, 2.0 ** -30, 2.0 ** 30) * np.where(
        np.arange(90) % 5 == 0, -1, 1)
    c["w"][7] = 0.0
    run_and_check(px, c, None, c["w"])
