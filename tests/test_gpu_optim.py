"""GPU parity of the global gradient norm, the clip and Adam over many tensors.

Bounds: the norm sums at most 34 squares in fp32 (each thread's share of a
chunk, relative error <= 36 2^-24) and the rest in 64 bits, so it is within
20 * 2^-24 relative, then rounded to fp32 (2^-24): 24 * 2^-24 in all.  A clipped element is
one product with the scale: the norm's error plus 2 * 2^-24 (fp32), and 2^-8
where the output is bf16.  Adam: the bound of the single call's parity test,
1e-5 relative plus 2e-7 of the array's largest magnitude (the first moment
cancels); clipped, the norm's 24 * 2^-24 = 1.4e-6 stays inside it.  The step
with unequal alignments gives the same bits as the aligned one."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block_oracle as bo  # noqa: E402
from tests.block_common import EPS, TDT, Guarded, host, status_ok, within  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM_REL = 24 * U

LISTS = [[1], [0, 5], [3, 0, 1, 0], [7] * 40, [8192, 8193, 1, 8191], [100000, 33, 262143],
         [4097] * 14, [5] * 1100, [2000001]]


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def make(counts, dtypes, seed, scale=1.0, shifts=(0,)):
    rng = np.random.default_rng(seed)
    g, grads, outs = Guarded(), [], []
    for i, n in enumerate(counts):
        d = TDT[dtypes[i % len(dtypes)]]
        t = g.tensor((n,), d, shifts[i % len(shifts)])
        t.copy_(torch.from_numpy(rng.standard_normal(n) * scale).to(d))
        grads.append(t)
        outs.append(g.tensor((n,), d, shifts[(i + 1) % len(shifts)]))
    return g, grads, outs


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16")])
@pytest.mark.parametrize("i", range(len(LISTS)))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_norm_and_clip(px, i, dtypes, max_norm):
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    shifts = (0,) if i % 2 else (0, 1, 3)
    g, grads, outs = make(LISTS[i], dtypes, 300 + i, shifts=shifts)
    before = [t.clone() for t in grads]
    clip = PoetxGradClip()
    h = [host(t) for t in grads]
    want = bo.grad_norm(h)
    assert abs(float(clip.total(grads)) - want) <= NORM_REL * want
    got = clip.clip(grads, max_norm, out=outs)
    status_ok(px)
    g.check()
    assert abs(float(got) - want) <= NORM_REL * want
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    _, ref = bo.clip(h, max_norm)
    for o, r in zip(outs, ref):
        if r.size:
            rel = NORM_REL + 2 * U + (EPS["bf16"] if o.dtype is torch.bfloat16 else 0)
            within(host(o), r, rel * np.abs(r))
    # in place: the same bits
    clip.clip(grads, max_norm)
    status_ok(px)
    g.check()
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
def test_squares_outside_fp32(px, scale, dtype):
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    g, grads, outs = make([5000, 17], (dtype,), 320, scale=scale)
    clip = PoetxGradClip()
    want = bo.grad_norm([host(t) for t in grads])
    assert abs(float(clip.clip(grads, 1e-3 * want, out=outs)) - want) <= NORM_REL * want
    g.check()
    got = bo.grad_norm([host(t) for t in outs])
    scaled = 1e-3 * want * want / (want + 1e-6) if 1e-3 * want < want + 1e-6 else want
    # elements below the smallest normal number are rounded to multiples of 2^-149 (bf16: 2^-133)
    under = (2.0 ** -149 if dtype == "f32" else 2.0 ** -133) * 5017 ** 0.5
    assert abs(got - scaled) <= (NORM_REL + EPS[dtype] + 4 * U) * scaled + under


def test_zeros_nan_inf_and_nothing(px):
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    clip = PoetxGradClip()
    a = torch.zeros(1000, device="cuda")
    assert float(clip.clip([a], 1.0)) == 0.0 and torch.count_nonzero(a) == 0
    assert float(clip.clip([], 1.0)) == 0.0
    assert float(clip.total([a[:0]])) == 0.0
    b = torch.ones(1000, device="cuda")
    b[7] = float("inf")
    assert float(clip.clip([b], 1.0)) == float("inf")
    assert torch.isnan(b[7]) and torch.count_nonzero(b[8:]) == 0  # 1 / inf = 0, inf * 0
    b = torch.ones(1000, device="cuda")
    b[999] = float("nan")
    assert np.isnan(float(clip.clip([a, b], 1.0))) and torch.isnan(b).all()
    b = torch.ones(4, device="cuda")
    clip.clip([b], 0.0)
    assert torch.count_nonzero(b) == 0
    clip.clip([b.fill_(2.0)], float("inf"))
    assert torch.all(b == 2.0)
    status_ok(px)


def f32(a):
    return float(np.float32(a))


HYPER = dict(lr=f32(1e-3), beta1=f32(0.9), beta2=f32(0.999), eps=f32(1e-8), weight_decay=f32(0.1))


def near(got, want):
    if want.size:
        within(host(got), want, 1e-5 * np.abs(want) + 2e-7 * np.abs(want).max())


@pytest.mark.parametrize("i", range(len(LISTS)))
@pytest.mark.parametrize("max_norm", [None, 0.5, 1e9])
def test_adam_matches_oracle(px, i, max_norm):
    import oracle
    from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam
    counts = LISTS[i]
    g, grads, _ = make(counts, ("f32",), 340 + i, shifts=(0,) if i % 2 else (0, 1, 3))
    _, theta, _ = make(counts, ("f32",), 360 + i, scale=0.1)
    opt = PoetxAdam([t.clone() for t in theta], lr=HYPER["lr"],
                    betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"],
                    weight_decay=HYPER["weight_decay"])
    want = [(host(t), np.zeros(n), np.zeros(n)) for t, n in zip(theta, counts)]
    g64 = [host(t) for t in grads]
    use = g64 if max_norm is None else bo.clip(g64, max_norm)[1]
    for step in (1, 2):
        opt.step(grads, max_norm=max_norm)
        want = [oracle.adam_update(*([t, gr, m, v, step]), **HYPER)
                for (t, m, v), gr in zip(want, use)]
    status_ok(px)
    g.check()
    for (t, m, v), p, om, ov in zip(want, opt.params, opt.m, opt.v):
        near(p, t), near(om, m), near(ov, v)
    assert opt.t == 2
    if max_norm is not None:
        norm = bo.grad_norm(g64)
        assert abs(float(opt.norm) - norm) <= NORM_REL * norm


def test_adam_takes_misaligned_vectors(px):
    n = 20011
    rng = np.random.default_rng(380)
    vals = [rng.standard_normal(n), rng.standard_normal(n), rng.standard_normal(n) * 0.1,
            rng.random(n)]
    got = []
    for shifts in ((0, 0, 0, 0), (0, 1, 2, 3), (3, 3, 3, 3), (1, 1, 2, 1)):
        g = Guarded()
        views = [g.tensor((n,), torch.float32, s) for s in shifts]
        for t, v in zip(views, vals):
            t.copy_(torch.from_numpy(v))
        th, gr, m, v = views
        px.poetx_adam_update_many([th], [gr], [m], [v], 3, 1e-2, weight_decay=0.5)
        status_ok(px)
        g.check()
        got.append([t.clone() for t in views])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_adam_list_in_several_launches_is_one_step(px):
    # more vectors than one launch's table holds: every vector gets its step, none twice
    from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam
    counts = [3 + i % 5 for i in range(1300)]
    _, grads, _ = make(counts, ("f32",), 385)
    whole = torch.cat([g.clone() for g in grads])
    a = PoetxAdam([torch.ones(n, device="cuda") for n in counts], lr=0.1)
    b = PoetxAdam([torch.ones(sum(counts), device="cuda")], lr=0.1)
    a.step(grads, max_norm=float("inf"))
    b.step([whole], max_norm=float("inf"))
    status_ok(px)
    assert torch.equal(torch.cat(a.params), b.params[0])


def test_same_bits_on_another_stream_and_in_a_graph(px):
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    _, grads, outs = make([50000, 3, 77777], ("f32", "bf16"), 390)
    clip = PoetxGradClip()
    clip.clip(grads, 0.5, out=outs)
    want = [t.clone() for t in outs] + [clip.norm.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    clip.clip(grads, 0.5, out=outs, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs + [clip.norm]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip.clip(grads, 0.5, out=outs)
    for o in outs:
        o.zero_()
    graph.replay()
    status_ok(px)
    assert all(torch.equal(a, b) for a, b in zip(want, outs + [clip.norm]))


def test_lists_are_checked(px):
    from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
    from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam
    a = torch.ones(8, device="cuda")
    clip = PoetxGradClip()
    for grads, kw in (([a.double()], {}), ([a[::2]], {}), ([a], {"out": [a[:4]]}),
                      ([a], {"out": [a, a]}), ([a], {"out": [a.bfloat16()]})):
        with pytest.raises(ValueError):
            clip.clip(grads, 1.0, **kw)
    with pytest.raises(px.PoetxError):
        clip.clip([a], -1.0)
    with pytest.raises(px.PoetxError):
        clip.clip([a], float("nan"))
    opt = PoetxAdam([a], lr=1e-3)
    for grads in ([a.bfloat16()], [a[:4]], [a, a], [torch.ones(16, device="cuda")[::2]]):
        with pytest.raises(ValueError):
            opt.step(grads, max_norm=1.0)
    with pytest.raises(ValueError):
        opt.step([a], max_norm=-2.0)
    assert opt.t == 0 and torch.all(a == 1)
