"""GPU parity of the matrix product with bias, activation and residual and of
its gradients, against the float64 oracle on the rounded inputs.

Bounds, per element.  A sum of K fp32 products in any order, rounded to
nearest or towards zero, is within K 2^-23 S of the exact one, S the sum of
the products' magnitudes (plus |bias|).  The activations have |act'| <= 1.13
(gelu_tanh's is the largest), and evaluate within 2^-18 (1 + |z|) in bf16 mode
(approximate exponential, argument and quotient errors of 2^-21 each; results
are then rounded to 2^-8) and 2^-21 (1 + |z|) in fp32 mode.  The result is
rounded once: u |y| with u = 2^-8 or 2^-24.  Backward: |act'(z)| evaluates
within the same absolute errors, so dz is within that times |dy|; bf16 rounds
dz once more (2^-8 |dz|) before the product, but not before dbias's sum."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block_oracle as bo  # noqa: E402
from tests.block_common import EPS, TDT, Guarded, host, rounded, status_ok, within  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
CODE = {n: i for i, n in enumerate(ACTS)}
ACT_ERR = {"bf16": 2.0 ** -18, "f32": 2.0 ** -21}

# (tokens, d_in, d_out): one token to several tiles, sizes on either side of
# the 16-, 64-, 128- and 256-wide tiles, odd ones, and single elements
SHAPES = [(1, 1, 1), (1, 64, 128), (1, 4096, 512), (2, 72, 40), (5, 3, 7), (7, 8, 8),
          (16, 256, 136), (17, 1000, 777), (24, 512, 1416), (33, 264, 1000), (64, 2048, 256),
          (65, 128, 520), (127, 192, 264), (128, 64, 128), (129, 320, 1288), (200, 576, 96),
          (256, 256, 256), (300, 136, 304), (513, 512, 640), (700, 1024, 2056), (1025, 2048, 513),
          # fp32: large enough for the tensor cores, either way
          (1301, 517, 1303), (900, 1536, 1200), (2100, 1000, 130), (700, 2056, 1024)]


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def dcode(px, dtype):
    return px.BF16 if dtype == "bf16" else px.F32


def inputs(T, a, b, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rounded(rng.standard_normal((T, a)), dtype)
    W = rounded(rng.standard_normal((b, a)) / np.sqrt(a), dtype)
    bias = rounded(rng.standard_normal(b) * 0.3, "f32")
    res = rounded(rng.standard_normal((T, b)), dtype)
    return x, W, bias, res


def forward_bounds(x, W, bias, z, y, dtype):
    S = np.abs(x) @ np.abs(W).T + (0 if bias is None else np.abs(bias))
    acc = (x.shape[1] + 2) * 2.0 ** -23 * S
    bz = acc + EPS[dtype] * (np.abs(z) + acc)
    by = 1.13 * acc + ACT_ERR[dtype] * (1 + np.abs(z)) + 2.0 ** -23 * np.abs(y)
    return by + EPS[dtype] * (np.abs(y) + by), bz


def run_forward(px, T, a, b, dtype, act, with_bias, with_res, with_z, seed, inplace=False):
    (x, x64), (W, W64), (bias, b64), (res, r64) = inputs(T, a, b, dtype, seed)
    if not with_bias:
        bias = b64 = None
    if not with_res:
        res = r64 = None
    g = Guarded()
    y = g.tensor((T, b), TDT[dtype])
    z = g.tensor((T, b), TDT[dtype]) if with_z else None
    ws = g.tensor((max(16, px.poetx_linear_forward_workspace_size(a, b, T, dcode(px, dtype))),),
                  torch.uint8)
    if inplace:
        y.copy_(res)
        res = y
    px.poetx_linear_forward(x, W, bias, res, y, z, a, b, T, CODE[act], dcode(px, dtype), ws)
    status_ok(px)
    g.check()
    want, zw = bo.linear(x64, W64, b64, r64, act)
    by, bz = forward_bounds(x64, W64, b64, zw, want, dtype)
    within(host(y), want, by, "y")
    if with_z:
        within(host(z), zw, bz, "z")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward_matches_oracle(px, i, dtype):
    # the options go round with the shapes, so that each is met in both types
    run_forward(px, *SHAPES[i], dtype, ACTS[i % 5], i % 2 == 0, i % 3 != 1, i % 4 < 2, 10 + i)


# Sizes that take each tile width, with whole and cut tiles and rows off 16 bytes,
# and the weight-streaming form with several tiles of tokens.
WIDTHS = [(1024, 72, 4096), (1000, 64, 4093), (1024, 72, 3648), (1001, 136, 3645),
          (2304, 64, 1536), (1000, 72, 1500), (260, 2048, 130), (600, 4096, 264)]


@pytest.mark.parametrize("i", range(len(WIDTHS)))
def test_every_tile_width(px, i):
    T, a, b = WIDTHS[i]
    run_forward(px, T, a, b, "bf16", ACTS[i % 5], i % 3 != 2, i % 2 == 0, i % 4 < 2, 110 + i)
    run_backward(px, T, b, a, "bf16", ACTS[(i + 1) % 5], True, i % 2 == 1, 130 + i)


# fp32 on the tensor cores, whose tiles are as wide as the rounds over the clusters ask for:
# 128 to 240 by 16 for the forward pass, by 32 for the backward one; 256
F32_WIDTHS = [(515, 2000), (1100, 2048), (1000, 3001), (515, 4100), (2048, 1500), (2048, 5000),
              (515, 5000), (1000, 4100), (300, 5000), (2048, 2048), (1280, 3800)]


@pytest.mark.parametrize("T,n", F32_WIDTHS)
def test_every_fp32_tile_width(px, T, n):
    run_forward(px, T, 320, n, "f32", "none", True, True, False, seed=n)
    run_backward(px, T, n, 320, "f32", "none", True, False, seed=T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,a,b", [(3, 128, 264), (150, 256, 384), (600, 512, 512)])
def test_every_activation_with_everything(px, T, a, b, act, dtype):
    run_forward(px, T, a, b, dtype, act, True, True, True, 50)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,a,b", [(1, 256, 256), (40, 128, 200), (300, 256, 512), (9, 33, 35)])
def test_residual_in_place(px, T, a, b, dtype):
    run_forward(px, T, a, b, dtype, "silu", False, True, False, 60, inplace=True)


def run_backward(px, T, a, b, dtype, act, want_dx, want_db, seed):
    rng = np.random.default_rng(seed)
    dy, dy64 = rounded(rng.standard_normal((T, b)) * 0.1, dtype)
    z, z64 = rounded(rng.standard_normal((T, b)) * 1.5, dtype)
    W, W64 = rounded(rng.standard_normal((b, a)) / np.sqrt(b), dtype)
    g = Guarded()
    dx = g.tensor((T, a), TDT[dtype]) if want_dx else None
    db = g.tensor((b,), torch.float32) if want_db else None
    ws = g.tensor((max(16, px.poetx_linear_backward_workspace_size(
        a, b, T, CODE[act], dcode(px, dtype), want_db)),), torch.uint8)
    px.poetx_linear_backward(dy, None if act == "none" else z, W, dx, db, a, b, T, CODE[act],
                             dcode(px, dtype), ws)
    status_ok(px)
    g.check()
    wx, wb, dz = bo.linear_backward(dy64, z64, W64, act)
    if want_db:
        bdz = ACT_ERR[dtype] * (1 + np.abs(z64)) * np.abs(dy64) if act != "none" else 0 * dz
        bb = bdz.sum(0) + (T + 2) * 2.0 ** -23 * np.abs(dz).sum(0)
        within(host(db), wb, bb + 2.0 ** -24 * np.abs(wb), "dbias")
    if want_dx:
        bdz = ACT_ERR[dtype] * (1 + np.abs(z64)) * np.abs(dy64) + EPS[dtype] * np.abs(dz)
        if act == "none":
            bdz = 0 * dz
        S = (np.abs(dz) + bdz) @ np.abs(W64)
        bx = bdz @ np.abs(W64) + (b + 2) * 2.0 ** -23 * S
        within(host(dx), wx, bx + EPS[dtype] * (np.abs(wx) + bx), "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward_matches_oracle(px, i, dtype):
    run_backward(px, *SHAPES[i], dtype, ACTS[(i + 2) % 5], True, i % 2 == 0, 90 + i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_backward_of_every_activation(px, act, dtype):
    run_backward(px, 300, 256, 512, dtype, act, True, True, 130)
    run_backward(px, 70, 40, 100, dtype, act, False, True, 131)


def test_dx_is_the_difference_of_the_forward(px):
    # fp32, through the library's own forward: d/dx of <dy, act(x W^T + b)> along a direction v,
    # (f(x + h v) - f(x - h v)) / 2h.  h = 2^-6: the third derivative's term is about
    # h^2 / 6 ~ 4e-5 of the sum's size, the fp32 rounding 2^-24 / h ~ 4e-6 of it
    T, a, b, act = 50, 96, 72, "gelu"
    (x, _), (W, _), (bias, _), _ = inputs(T, a, b, "f32", 140)
    rng = np.random.default_rng(141)
    dy, dy64 = rounded(rng.standard_normal((T, b)), "f32")
    v, v64 = rounded(rng.standard_normal((T, a)), "f32")
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(a, b, T, act=act, dtype="f32", save_z=True, backward=True)
    h = 2.0 ** -6
    up = host(layer.forward(x + h * v, W, bias))
    down = host(layer.forward(x - h * v, W, bias))
    want = float((dy64 * (up - down)).sum() / (2 * h))
    layer.forward(x, W, bias)
    dx, dbias = layer.backward(dy, W)
    got = float((host(dx) * v64).sum())
    scale = float(np.linalg.norm(dy64) * np.linalg.norm((up - down) / (2 * h)))
    assert abs(got - want) <= 1e-3 * scale
    assert abs(float(host(dbias) @ np.ones(b))) > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,a,b", [(20, 64, 128), (300, 256, 512), (1301, 517, 1303)])
def test_nan_and_inf_stay_in_their_token(px, T, a, b, dtype):
    (x, _), (W, _), (bias, _), (res, _) = inputs(T, a, b, dtype, 150)
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(a, b, T, act="relu", dtype=dtype, save_z=True)
    clean = layer.forward(x, W, bias, res).clone()
    x[3, 5] = float("nan")
    x[T - 1, 0] = float("inf")
    y = layer.forward(x, W, bias, res)
    status_ok(px)
    assert torch.isnan(y[3]).all()
    assert not torch.isfinite(layer.z[T - 1]).any()
    keep = [t for t in range(T) if t not in (3, T - 1)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T,a,b", [(700, 4096, 1024), (1301, 517, 1303), (900, 1536, 1200)])
def test_fp32_keeps_its_accuracy_on_the_tensor_cores(px, T, a, b):
    # Sums over 128 of K truncate at eight steps, each by at most 2^-23 and half of it on
    # average, so the whole by 8 * 2^-24 = 4.8e-7 on average; the fp32 additions of the partial
    # sums round to nearest (2^-24 each, of either sign).  Twice the average: 1e-6.
    (x, x64), (W, W64), _, _ = inputs(T, a, b, "f32", 180)
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(a, b, T, dtype="f32", backward=True)
    want = x64 @ W64.T
    assert np.linalg.norm(host(layer.forward(x, W)) - want) <= 1e-6 * np.linalg.norm(want)
    dy, dy64 = rounded(np.random.default_rng(181).standard_normal((T, b)), "f32")
    want = dy64 @ W64
    dx, _ = layer.backward(dy, W)
    status_ok(px)
    assert np.linalg.norm(host(dx) - want) <= 1e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e15, 1e38])
def test_fp32_over_its_whole_range(px, scale):
    # values whose bf16 planes under- or overflow: large x with small W and the other way round
    T, a, b = 1301, 517, 1303
    rng = np.random.default_rng(190)
    x, x64 = rounded(rng.uniform(1, 3.3, (T, a)) * scale, "f32")
    W, W64 = rounded(rng.standard_normal((b, a)) / scale * 1e-2, "f32")
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    y = host(PoetxLinear(a, b, T, dtype="f32").forward(x, W))
    status_ok(px)
    S = np.abs(x64) @ np.abs(W64).T
    # subnormal parts (below 2^-126) may be lost whole: 517 of them times the largest factor
    lost = 517 * 2.0 ** -126 * max(np.abs(x64).max(), np.abs(W64).max())
    within(y, x64 @ W64.T, (a + 4) * 2.0 ** -23 * S + lost)


def test_zero_tokens(px):
    W = torch.zeros((64, 32), dtype=torch.bfloat16, device="cuda")
    db = torch.full((64,), 7.0, device="cuda")
    px.poetx_linear_forward(None, W, None, None, None, None, 32, 64, 0, 0, px.BF16, None)
    px.poetx_linear_backward(None, None, W, None, db, 32, 64, 0, 0, px.BF16, None)
    status_ok(px)
    assert torch.count_nonzero(db) == 0


@pytest.mark.parametrize("dtype,T,a,b", [("bf16", 1, 512, 512), ("bf16", 40, 1024, 264),
                                         ("bf16", 900, 512, 768), ("f32", 200, 136, 264),
                                         ("f32", 1301, 517, 1303)])
def test_same_bits_on_another_stream_and_in_a_graph(px, dtype, T, a, b):
    (x, _), (W, _), (bias, _), (res, _) = inputs(T, a, b, dtype, 160)
    dy, _ = rounded(np.random.default_rng(161).standard_normal((T, b)), dtype)
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(a, b, T, act="silu", dtype=dtype, save_z=True, backward=True)

    def step(stream=None):
        layer.forward(x, W, bias, res, stream=stream)
        layer.backward(dy, W, stream=stream)

    def outputs():
        return [t.clone() for t in (layer.y, layer.z, layer.dx, layer.dbias)]

    step()
    want = outputs()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(outputs(), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (layer.y, layer.z, layer.dx, layer.dbias):
        t.zero_()
    graph.replay()
    status_ok(px)
    assert all(torch.equal(p, q) for p, q in zip(outputs(), want))


def test_fewer_tokens_than_the_layer_holds(px):
    (x, x64), (W, W64), _, _ = inputs(9, 64, 128, "bf16", 170)
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(64, 128, 32)
    y = layer.forward(x, W)
    assert y.shape == (9, 128)
    want, z = bo.linear(x64, W64, None, None, "none")
    within(host(y), want, forward_bounds(x64, W64, None, z, want, "bf16")[0])
    with pytest.raises(ValueError):
        PoetxLinear(64, 128, 4).forward(x, W)
    with pytest.raises(ValueError):
        layer.forward(x.t(), W)
    with pytest.raises(RuntimeError):
        layer.backward(y, W)
