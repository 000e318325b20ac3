"""Host-side checks of the head's losses (no GPU needed): workspace sizes, and what
the calls and classes refuse before anything is enqueued."""

import ctypes

import pytest
import torch

import orthogonal_reparameterized_packed_gb300 as poetx
from orthogonal_reparameterized_packed_gb300.build import build_library

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
B, F = poetx.BF16, poetx.F32
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    build_library()
    return poetx.load_library()


def test_workspaces(L):
    for size in (lambda *a: L.poetx_cross_entropy_workspace_size(*a),
                 lambda d, v, t, *a: L.poetx_distill_workspace_size(d, v, t, 8, *a)):
        for dt in (B, F):
            assert size(64, 1000, 40, dt, 3, 0) > 0
            for bad in ((0, 1000, 40, dt, 3, 0), (64, 0, 40, dt, 3, 0), (64, 1000, -1, dt, 3, 0),
                        (64, 1000, 40, 7, 3, 0), (64, 1000, 40, dt, 4, 0),
                        (64, 1000, 40, dt, -1, 0), (64, 1000, 40, dt, 3, -1),
                        ((1 << 20) + 1, 1000, 40, dt, 3, 0), (64, (1 << 20) + 1, 40, dt, 3, 0),
                        (64, 1000, (1 << 22) + 1, dt, 3, 0), (64, 1000, 0, dt, 3, 0)):
                assert size(*bad) == 0, bad
    assert L.poetx_distill_workspace_size(64, 1000, 40, 0, B, 0, 0) == 0
    assert L.poetx_distill_workspace_size(64, 1000, 40, 1025, B, 0, 0) == 0


@pytest.mark.parametrize("dt", [B, F])
@pytest.mark.parametrize("grads", [0, 1, 2, 3])
@pytest.mark.parametrize("block", [0, 64, 300])
def test_the_workspace_of_more_tokens_is_enough_for_fewer(L, dt, grads, block):
    for d, V in ((64, 1000), (65, 777), (256, 6400), (1024, 300), (2048, 2000)):
        last = 0
        for t in (1, 2, 17, 63, 64, 65, 128, 129, 255, 256, 257, 300, 511, 513, 1000, 1025, 2048,
                  2049, 5000, 8192):
            n = L.poetx_cross_entropy_workspace_size(d, V, t, dt, grads, block)
            assert n >= last, (d, V, t)
            last = n


def test_the_workspace_is_bounded(L):
    """A block's terms, not the logits: 2 GiB beside what grows with the tokens' rows, and
    for several blocks with dW the head in fp32."""
    d, V = 2048, 128000
    for t in (8192, 65536, 1 << 20):
        rows = t * (4 * d + 256) + (64 << 20)
        for dt in (B, F):
            planes = 3 * 2 * (V * d + 16384 * V) * (dt == F) + 2 * (t * d * 6) * (dt == F)
            assert L.poetx_cross_entropy_workspace_size(d, V, t, dt, 1, 0) <= (
                (2 << 30) + (1 << 29) + rows + planes)


def test_cross_entropy_rejects_invalid_arguments(L):
    need = L.poetx_cross_entropy_workspace_size(64, 1000, 40, B, 3, 0)

    def call(x=FAKE, W=2 * FAKE, y=3 * FAKE, size=8, w=4 * FAKE, loss=5 * FAKE, total=6 * FAKE,
             dx=7 * FAKE, dW=8 * FAKE, d=64, V=1000, T=40, dt=B, block=0, work=FAKE, n=BIG):
        return L.poetx_cross_entropy(x, W, y, size, w, loss, total, dx, dW, d, V, T, dt, block,
                                     work, n, None)

    bad = [dict(x=None), dict(W=None), dict(y=None), dict(loss=None), dict(total=None),
           dict(size=2), dict(size=0), dict(x=FAKE + 8), dict(W=FAKE + 2), dict(y=FAKE + 4),
           dict(y=FAKE + 2, size=4), dict(w=FAKE + 2), dict(loss=FAKE + 1), dict(total=FAKE + 2),
           dict(dx=FAKE + 8), dict(dW=FAKE + 4), dict(dx=FAKE), dict(dx=2 * FAKE), dict(dW=FAKE),
           dict(dW=2 * FAKE), dict(dW=7 * FAKE), dict(d=0), dict(V=-1), dict(T=-1),
           dict(T=(1 << 22) + 1), dict(d=(1 << 20) + 1), dict(V=(1 << 20) + 1), dict(dt=2),
           dict(block=-1), dict(block=(1 << 22) + 1), dict(w=5 * FAKE)]
    for kw in bad:
        assert call(**kw) == 1, kw
    assert call(n=need - 1) == 3 and call(work=None) == 3 and call(work=FAKE + 8) == 3


def test_distill_rejects_invalid_arguments(L):
    f = ctypes.c_float
    need = L.poetx_distill_workspace_size(64, 1000, 40, 8, B, 0, 0)

    def call(x=FAKE, W=2 * FAKE, i=3 * FAKE, size=4, s=9 * FAKE, sdt=F, w=None, loss=5 * FAKE,
             total=6 * FAKE, dx=None, dW=None, d=64, V=1000, T=40, top=8, tau=2.0, dt=B, block=0,
             work=FAKE, n=BIG):
        return L.poetx_distill(x, W, i, size, s, sdt, w, loss, total, dx, dW, d, V, T, top, f(tau),
                               dt, block, work, n, None)

    bad = [dict(i=None), dict(s=None), dict(sdt=2), dict(sdt=-1), dict(s=FAKE + 2),
           dict(s=FAKE + 1, sdt=B), dict(top=0), dict(top=-1), dict(top=1025), dict(tau=0.0),
           dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=65.0),
           dict(tau=0.01), dict(size=1), dict(i=FAKE + 2), dict(d=0), dict(T=-1)]
    for kw in bad:
        assert call(**kw) == 1, kw
    assert call(n=need - 1) == 3


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU, for checks that come before any use."""

    is_cuda = True


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    """Objects on the host whose calls end in a list."""
    from orthogonal_reparameterized_packed_gb300 import loss
    got = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: got.append((name, a)) or 0

    monkeypatch.setattr(loss, "load_library", Lib)
    monkeypatch.setattr(loss, "poetx_cross_entropy_workspace_size", lambda *a: 64)
    monkeypatch.setattr(loss, "poetx_distill_workspace_size", lambda *a: 64)
    monkeypatch.setattr(loss, "_stream", lambda s: 0)
    return got


def test_classes_refuse_what_the_kernels_would_read_wrongly(calls):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    kw = dict(device="cpu", backward=True, weight_grad=True)
    ce = PoetxCrossEntropy(16, 50, 8, **kw)
    kd = PoetxDistill(16, 50, 8, top=3, temperature=2.0, **kw)
    x, W, w = on_gpu(8, 16), on_gpu(50, 16), on_gpu(8, dtype=torch.float32)
    y = on_gpu(8, dtype=torch.int64)
    idx, s = on_gpu(8, 3, dtype=torch.int32), on_gpu(8, 3, dtype=torch.float32)
    for args in ((on_gpu(9, 16), W, on_gpu(9, dtype=torch.int64)), (on_gpu(8, 15), W, y),
                 (x.float(), W, y), (torch.zeros(8, 16).bfloat16(), W, y),
                 (on_gpu(8, 32)[:, ::2], W, y), (x, on_gpu(49, 16), y), (x, W.float(), y),
                 (x, W, y[:7]), (x, W, y.float()), (x, W, y.short()),
                 (x, W, on_gpu(8, 2, dtype=torch.int64)[:, 0]), (x, W, torch.zeros(8).long()),
                 (x, W, y, w.bfloat16()), (x, W, y, w[:7]), (x, W, y, torch.ones(8))):
        for call in (ce.forward, ce.step):
            with pytest.raises(ValueError):
                call(*args)
    for args in ((x, W, idx[:, :2], s[:, :2]), (x, W, idx, s[:, :2]), (x, W, idx, s.half()),
                 (x, W, idx, s.double()), (x, W, idx.float(), s), (x, W, idx.t(), s.t()),
                 (x, W, idx, torch.zeros(8, 3)), (x, W, idx[:7], s), (x, W, idx, s, w[1:])):
        for call in (kd.forward, kd.step):
            with pytest.raises(ValueError):
                call(*args)
    assert calls == []
    ce.step(x, W, y, w)
    kd.step(x[:5], W, idx[:5], s[:5])
    kd.forward(x, W, idx.long(), s.bfloat16())
    assert [n for n, _ in calls] == ["poetx_cross_entropy", "poetx_distill", "poetx_distill"]


def test_classes_refuse_what_they_were_not_made_for(calls, monkeypatch, L):
    from orthogonal_reparameterized_packed_gb300 import loss as loss_module
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    x, W, y = on_gpu(8, 16), on_gpu(50, 16), on_gpu(8, dtype=torch.int64)
    with pytest.raises(RuntimeError):
        PoetxCrossEntropy(16, 50, 8, device="cpu").step(x, W, y)
    with pytest.raises(ValueError):
        PoetxCrossEntropy(16, 50, 8, device="cpu", weight_grad=True)
    for block in (0, -1):
        with pytest.raises(ValueError):
            PoetxDistill(16, 50, 8, top=2, device="cpu", block_tokens=block)
    monkeypatch.setattr(loss_module, "poetx_distill_workspace_size",
                        poetx.poetx_distill_workspace_size)
    for top in (0, 1025):
        with pytest.raises(ValueError, match="limits"):
            PoetxDistill(16, 50, 8, top=top, device="cpu")
    loss, dx, dW = PoetxCrossEntropy(16, 50, 8, device="cpu", backward=True).step(x, W, y)
    assert dW is None and calls[0][1][8] is None


def test_tensors_of_another_device_are_refused(calls, monkeypatch):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy
    ce = PoetxCrossEntropy(16, 50, 8, device="cpu")
    ce._device = 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(OnGpu, "get_device", lambda self: 0, raising=False)
    x, W, y = on_gpu(8, 16), on_gpu(50, 16), on_gpu(8, dtype=torch.int64)
    with pytest.raises(ValueError, match="current device"):
        ce.forward(x, W, y)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ce.forward(x, W, y)
    monkeypatch.setattr(OnGpu, "get_device", lambda self: 1, raising=False)
    with pytest.raises(ValueError, match="tensors on"):
        ce.forward(x, W, y)
    assert len(calls) == 1
