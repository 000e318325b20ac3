"""Edges of the operators around the projections: what one call reads of the
one before it in its stream."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.block_common import status_ok  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def normal(*shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,a,b", [(300, 256, 520), (1100, 512, 768)])
def test_dbias_of_gradients_written_just_before(px, T, a, b, dtype):
    # 60 backward passes in a row through one workspace, each of values that a kernel writes
    # right before it: the bits of the same passes one by one
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    n, layer = 60, PoetxLinear(a, b, T, act="silu", dtype=dtype, backward=True)
    W, dy, z = (normal(*s, seed=400 + i).to(layer.dtype) * 0.1
                for i, s in enumerate(((b, a), (T, b), (T, b))))
    now = torch.empty_like(dy)

    def one(i):
        torch.mul(dy, 1.0 + i, out=now)
        dx, dbias = layer.backward(now, W, z=z)
        return dx.clone(), dbias.clone()

    want = []
    for i in range(n):
        want.append(one(i))
        torch.cuda.synchronize()
    got = [one(i) for i in range(n)]
    status_ok(px)
    for i in range(n):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i])), i
    assert len({float(w[1].double().sum()) for w in want}) == n


@pytest.mark.parametrize("counts", [[5000, 3, 700], [8192] * 30, [20000] * 90])
def test_clip_of_gradients_written_just_before(px, counts):
    # 100 clips in a row, lists from fewer chunks than SMs on, each of values that a kernel
    # writes right before it: the bits of the same clips one by one
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    n, clip = 100, PoetxGradClip()
    base = normal(sum(counts), seed=410)
    now, out = torch.empty_like(base), torch.empty_like(base)
    grads, outs = now.split(counts), out.split(counts)

    def one(i):
        torch.mul(base, 1.0 + i, out=now)
        norm = clip.clip(grads, 0.5, out=outs)
        return out.clone(), norm.clone()

    want = []
    for i in range(n):
        want.append(one(i))
        torch.cuda.synchronize()
    got = [one(i) for i in range(n)]
    status_ok(px)
    for i in range(n):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i])), i
    assert len({float(w[1]) for w in want}) == n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D", [(1, 128), (1, 96), (2, 64)])
def test_every_group_of_heads_begins_a_token(px, heads, D, dtype):
    # one group of heads per token: every step of a warp takes the table's next row into the
    # ring and reads the one before; the bits of the same tokens in one call of their own
    from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope, rope_tables
    T = 9001
    cos, sin = rope_tables(T, D)
    q, dq = (normal(T, heads * D, seed=420 + i) for i in range(2))
    q, dq = (t.to(torch.bfloat16) if dtype == "bf16" else t for t in (q, dq))
    none = q[:, :0]
    step = PoetxQKNormRope(heads, 0, D, T, dtype=dtype, backward=True)
    y = step.forward(q, none, None, None, cos, sin)[0].clone()
    dx = step.backward(dq, none, q, none, None, None, cos, sin)[0].clone()
    at = torch.arange(T, dtype=torch.int32, device="cuda")
    for t0 in range(0, T, 700):
        s = slice(t0, min(T, t0 + 700))
        assert torch.equal(step.forward(q[s], none, None, None, cos, sin, at[s])[0], y[s])
        assert torch.equal(step.backward(dq[s], none, q[s], none, None, None, cos, sin,
                                         at[s])[0], dx[s])
    status_ok(px)


# (tokens, d_in, d_out) for which a product of these tokens takes more scratch than one of
# tokens + 1 (tensor cores with 256 tokens, CUDA cores with 257)
STEPS = [(256, 256, 6400), (256, 256, 6144), (512, 256, 6400), (300, 1000, 2000)]


@pytest.mark.parametrize("T,a,b", STEPS)
def test_fp32_layer_takes_fewer_tokens_than_it_holds(px, T, a, b):
    # results are those of a layer made for the tokens, both ways, at every capacity
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    x, W = normal(T, a, seed=430), normal(b, a, seed=431, scale=a ** -0.5)
    dy, V = normal(T, a, seed=432), normal(a, b, seed=433, scale=b ** -0.5)
    want = PoetxLinear(a, b, T, dtype="f32").forward(x, W)
    back = [t.clone() for t in PoetxLinear(b, a, T, dtype="f32", backward=True).backward(dy, V)]
    for more in (1, 2, 40, 1000):
        layer = PoetxLinear(a, b, T + more, dtype="f32")
        assert torch.equal(layer.forward(x, W), want)
        layer = PoetxLinear(b, a, T + more, dtype="f32", backward=True)
        assert all(torch.equal(p, q) for p, q in zip(layer.backward(dy, V), back))
    status_ok(px)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("a,b", [(256, 6400), (6400, 256), (5120, 320), (78, 3050), (147, 1098),
                                 (1000, 999), (4096, 4096), (33, 7)])
def test_workspace_of_more_tokens_serves_fewer(px, a, b, dtype):
    code = px.BF16 if dtype == "bf16" else px.F32
    for size in (lambda t: px.poetx_linear_forward_workspace_size(a, b, t, code),
                 lambda t: px.poetx_linear_backward_workspace_size(a, b, t, 2, code),
                 lambda t: px.poetx_linear_backward_workspace_size(a, b, t, 0, code, False)):
        sizes = [size(t) for t in [*range(1, 1100), 5000, 5001, 1 << 20, 1 << 22]]
        assert all(p <= q for p, q in zip(sizes, sizes[1:]))


def through_identity(px, dtype, act, z, dy, sums=True):
    """(dx, dbias) of a layer with the unit weight: dz itself, rounded, and its sums."""
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    T, n = z.shape
    layer = PoetxLinear(n, n, T, act=act, dtype=dtype, backward=True)
    dx, dbias = layer.backward(dy, torch.eye(n, device="cuda", dtype=layer.dtype), z=z)
    status_ok(px)
    return dx, dbias


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n", [(5, 64), (70, 72), (1000, 520)])
def test_relu_passes_no_gradient_where_it_is_zero(px, T, n, dtype):
    # infinite and NaN gradients at z <= 0 and at NaN: dz = 0 there, as the definition selects
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z, dy = normal(T, n, seed=440).to(tdt), normal(T, n, seed=441).to(tdt)
    z[0, 1], z[1, 2], z[T - 1, n - 1] = 0.0, float("-inf"), float("nan")
    off = ~(z > 0)
    want = torch.where(off, torch.zeros_like(dy), dy)
    for bad in (float("inf"), float("-inf"), float("nan")):
        spoilt = torch.where(off, torch.full_like(dy, bad), dy)
        dx, dbias = through_identity(px, dtype, "relu", z, spoilt)
        assert torch.equal(dx, want)
        clean = through_identity(px, dtype, "relu", z, want)[1]
        assert torch.equal(dbias, clean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_gradient_of_large_finite_values(px, act, dtype):
    # far from zero every activation's slope is 1 or 0, whatever leaves the range on the way
    # (silu's and gelu's slope is 1 + z e^-z .. there: within 1e-40 of 1 from z = 100 on)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    top = float(torch.finfo(tdt).max)
    z = torch.tensor([1e2, 1e4, 1e10, 1e18, 1.9e19, 1e20, 1e30, top], device="cuda").repeat(5, 8)
    for sign, slope in ((1, 1.0), (-1, 0.0)):
        dx, dbias = through_identity(px, dtype, act, (sign * z).to(tdt),
                                     torch.ones_like(z).to(tdt))
        assert torch.all(dx == slope) and torch.all(dbias == 5 * slope)


def test_gelu_is_relatively_accurate_in_its_tail(px):
    # bf16: z Phi(z) from -0.5 down to where it leaves bf16's normal range, through the unit
    # weight.  Phi's approximation is within 2^-13 relative, its exponential within
    # |z^2 / 2| 2^-23 of argument and quotient errors (2^-16 at z = -12.5), the result is
    # rounded once (2^-8); z + 0 is exact.
    from math import erfc
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    n = 64
    for T in (16, 1000):
        x = torch.linspace(-12.5, -0.5, T * n, device="cuda").view(T, n).bfloat16()
        layer = PoetxLinear(n, n, T, act="gelu")
        y = layer.forward(x, torch.eye(n, device="cuda", dtype=torch.bfloat16))
        status_ok(px)
        x64 = x.double().cpu().numpy()
        want = x64 * 0.5 * np.vectorize(erfc)(-x64 / np.sqrt(2))
        off = np.abs(y.double().cpu().numpy() / want - 1)
        assert off.max() <= 2.0 ** -8 + 2.0 ** -12, (off.max(), x64.flat[off.argmax()])


def fp32_product(px, x, W, residual=None, inplace=False):
    """x W^T (+ residual) and the magnitudes' sums, in 64 bits too."""
    from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
    layer = PoetxLinear(x.shape[1], W.shape[0], x.shape[0], dtype="f32")
    y = layer.forward(x, W, residual=residual)
    status_ok(px)
    x64, W64 = x.double().cpu().numpy(), W.double().cpu().numpy()
    return y.double().cpu().numpy(), x64 @ W64.T, np.abs(x64) @ np.abs(W64).T


# fp32 sizes of the tensor cores, [N][K] weights
LARGE = [(1301, 517, 1303), (700, 2056, 1024)]


@pytest.mark.parametrize("T,a,b", LARGE)
@pytest.mark.parametrize("exponent", [-126, -120, -114, -110, -109, -108, -100, -60, 59, 61, 80])
def test_fp32_rows_of_any_size_keep_24_bits(px, T, a, b, exponent):
    # a few tokens of this size among others of size 1, weights of the opposite size, so that
    # no product leaves the normal range; K 2^-23 of the magnitudes' sum, as every fp32 sum
    x, W = normal(T, a, seed=450), normal(b, a, seed=451, scale=a ** -0.5)
    far = [0, 3, T // 2, T - 1]
    x[far] = torch.rand((len(far), a), device="cuda") * 2.0 ** exponent + 2.0 ** exponent
    if abs(exponent) > 100:
        W *= 2.0 ** 40
    y, want, S = fp32_product(px, x, W)
    assert np.all(np.abs(y - want) <= (a + 4) * 2.0 ** -23 * S)
    # far fewer bits would be lost than the bound allows: also on the average of a row
    for t in far:
        assert np.linalg.norm(y[t] - want[t]) <= 1e-6 * np.linalg.norm(want[t])


@pytest.mark.parametrize("T,a,b", LARGE)
def test_fp32_weights_of_any_size_keep_24_bits(px, T, a, b):
    x, W = normal(T, a, seed=452), normal(b, a, seed=453)
    for small in (1.5e-38, 3e-34, 5e19):
        V = W.clone()
        V[7] *= small
        y, want, S = fp32_product(px, x, V)
        assert np.all(np.abs(y - want) <= (a + 4) * 2.0 ** -23 * S + a * 2.0 ** -149)


@pytest.mark.parametrize("T,a,b", LARGE)
def test_fp32_products_beyond_the_range_are_infinite(px, T, a, b):
    # one product each of a sign, far beyond fp32, in values just under a bf16 number (whose
    # second parts have the other sign); the rest of the row is small
    x, W = normal(T, a, seed=454), normal(b, a, seed=455)
    x[5, 9] = 3e38 * (1 - 2.0 ** -12)
    W[:, 9] = W[:, 9].sign() * 1e6 * (1 - 2.0 ** -12)
    x[:, 9].mul_((torch.arange(T, device="cuda") == 5).float())
    y, want, _ = fp32_product(px, x, W)
    assert np.array_equal(y[5], np.sign(W[:, 9].double().cpu().numpy()) * np.inf)
    keep = [t for t in range(T) if t != 5]
    assert np.isfinite(y[keep]).all()


@pytest.mark.parametrize("T,a,b", LARGE)
def test_fp32_products_near_the_bottom_of_the_range(px, T, a, b):
    # both operands inside what the tensor cores take, products of 2^-120: each of the six sums
    # of a product's parts is rounded to a multiple of 2^-149, and truncated up to once more
    x, W = normal(T, a, seed=456) * 2.0 ** -70, normal(b, a, seed=457) * 2.0 ** -50
    y, want, S = fp32_product(px, x, W)
    bottom = 12 * a * 2.0 ** -149
    assert np.all(np.abs(y - want) <= (a + 4) * 2.0 ** -23 * S + bottom)
    assert np.linalg.norm(y - want) <= 1e-6 * np.linalg.norm(want) + bottom * want.size ** 0.5


def test_no_key_heads_have_no_gradient(px):
    # dgamma_k of a step without key heads: the sum over no rows, not what the memory held
    from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope, rope_tables
    D, T = 64, 20
    stale = [torch.full((D,), 7.0, device="cuda") for _ in range(8)]
    del stale
    step = PoetxQKNormRope(2, 0, D, T, dtype="f32", backward=True)
    q, dq = normal(T, 2 * D, seed=460), normal(T, 2 * D, seed=461)
    dk, dgamma_k = step.backward(dq, dq[:, :0], q, q[:, :0], None, None,
                                 *rope_tables(T, D))[1::2]
    status_ok(px)
    assert dk.shape == (T, 0) and dgamma_k.shape == (D,)
    assert torch.count_nonzero(dgamma_k) == 0


def test_one_clip_on_two_streams_at_one_time(px):
    # long and short lists on two streams, many times with nothing between: every norm and
    # every output has the bits of a call on its own
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    counts = ([60000] * 40, [500, 7])
    sides, clip = [torch.cuda.Stream() for _ in counts], PoetxGradClip()
    grads = [[normal(n, seed=470 + 50 * i + j) for j, n in enumerate(c)]
             for i, c in enumerate(counts)]
    outs = [[torch.empty_like(g) for g in gs] for gs in grads]
    want = []
    for g, o in zip(grads, outs):
        norm = clip.clip(g, 0.5, out=o)
        torch.cuda.synchronize()
        want.append((norm.clone(), [t.clone() for t in o]))
    torch.cuda.synchronize()
    for _ in range(50):
        norms = [clip.clip(g, 0.5, out=o, stream=s) for g, o, s in zip(grads, outs, sides)]
    status_ok(px)
    for (norm, values), got, o in zip(want, norms, outs):
        assert torch.equal(got, norm) and all(torch.equal(p, q) for p, q in zip(o, values))
