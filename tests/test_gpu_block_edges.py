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
