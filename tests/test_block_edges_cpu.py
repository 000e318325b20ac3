"""Host-side edges of the operators around the projections (no GPU needed):
what the calls and classes refuse before anything is enqueued."""

import ctypes

import pytest
import torch

import orthogonal_reparameterized_packed_gb300 as poetx
from orthogonal_reparameterized_packed_gb300.build import build_library

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
B = poetx.BF16


@pytest.fixture(scope="module")
def L():
    build_library()
    return poetx.load_library()


def test_linear_forward_needs_its_workspace(L):
    # rows of 65 bf16 features are copied to aligned ones first
    need = poetx.poetx_linear_forward_workspace_size(65, 128, 40, B)
    assert need > 0

    def fwd(work=FAKE, n=need):
        return L.poetx_linear_forward(FAKE, FAKE, None, None, FAKE + 4096, None, 65, 128, 40, 0, B,
                                      work, n, None)

    assert fwd(n=need - 1) == 3 and fwd(work=None) == 3 and fwd(work=FAKE + 8) == 3


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU, for checks that come before any use."""

    is_cuda = True


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    """In the library's place: what reached it; every call returns POETX_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 64

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    # on these host tensors nothing may be launched: the calls end here
    fake = Recorder()
    monkeypatch.setattr(poetx, "load_library", lambda: fake)
    monkeypatch.setattr(poetx, "_stream", lambda stream: 0)
    return fake


def test_lists_of_the_calls_go_together(lib):
    a, b, h = on_gpu(8), on_gpu(6), on_gpu(8, dtype=torch.bfloat16)
    norm, ws = on_gpu(1), on_gpu(16)
    host, strided, double = torch.zeros(8), on_gpu(8, 2)[:, 0], on_gpu(8, dtype=torch.float64)
    for grads in ([host], [strided], [double], [a, host]):
        with pytest.raises(ValueError):
            poetx.poetx_grad_norm(grads, norm, ws)
        with pytest.raises(ValueError):
            poetx.poetx_clip_grads(grads, None, 1.0, norm, ws)
    for outs in ([], [a], [a, a], [b, a], [a, b, a], [h, b], [host, b], [strided, b]):
        with pytest.raises(ValueError):
            poetx.poetx_clip_grads([a, b], outs, 1.0, norm, ws)
    good = [a, b]
    for bad in ([], [a], [a, a], [b, a], [a, b, b], [h, b], [host, b], [strided, b]):
        for i in range(4):
            lists = [good] * 4
            lists[i] = bad
            with pytest.raises(ValueError):
                poetx.poetx_adam_update_many(*lists, 1, 1e-3)
    assert lib.calls == []
    poetx.poetx_clip_grads([a, h], [a, h], 1.0, norm, ws)
    poetx.poetx_adam_update_many(good, good, good, good, 1, 1e-3)
    assert [n for n, _ in lib.calls] == ["poetx_clip_grads", "poetx_adam_update_many"]


def test_lists_may_be_any_iterable(lib):
    a, b, norm, ws = on_gpu(8), on_gpu(6), on_gpu(1), on_gpu(16)
    poetx.poetx_grad_norm((t for t in (a, b)), norm, ws)
    poetx.poetx_clip_grads((t for t in (a, b)), iter([a, b]), 1.0, norm, ws)
    poetx.poetx_adam_update_many(*[(t for t in (a, b)) for _ in range(4)], 1, 1e-3)
    assert [args[0] for _, args in lib.calls] == [2, 2, 2]


BAD = [torch.zeros(8),                                 # on the host
       on_gpu(8, 2)[:, 0],                             # every other element
       on_gpu(4, 2).t(),                               # dense, in another order
       on_gpu(8, dtype=torch.bfloat16), on_gpu(8, dtype=torch.float64)]


def test_adam_refuses_parameters_that_it_would_read_wrongly(lib):
    from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam
    for bad in BAD:
        with pytest.raises(ValueError):
            PoetxAdam([on_gpu(3), bad], lr=1e-3)
    assert lib.calls == []


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_adam_refuses_gradients_and_moments_that_do_not_fit(lib, monkeypatch, max_norm):
    from orthogonal_reparameterized_packed_gb300 import layer
    monkeypatch.setattr(layer, "poetx_grad_norm_workspace_size", lambda n: 64)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: on_gpu(64))
    opt = layer.PoetxAdam([on_gpu(8), on_gpu(6)], lr=1e-3)
    good = [on_gpu(8), on_gpu(6)]
    for bad in [*([b, good[1]] for b in BAD), [on_gpu(7), good[1]], [good[1], good[0]]]:
        with pytest.raises(ValueError):
            opt.step(bad, max_norm=max_norm)
    for name in ("params", "m", "v"):
        for bad in [*([b, good[1]] for b in BAD), good[:1], [*good, good[0]], [good[1], good[0]]]:
            kept = getattr(opt, name)
            setattr(opt, name, bad)
            with pytest.raises(ValueError):
                opt.step(good, max_norm=max_norm)
            setattr(opt, name, kept)
    opt.m[1] = on_gpu(5)  # in place too
    with pytest.raises(ValueError):
        opt.step(good, max_norm=max_norm)
    opt.m[1] = on_gpu(6)
    assert lib.calls == [] and opt.t == 0
    opt.step((g for g in good), max_norm=max_norm)
    assert opt.t == 1 and len(lib.calls) == (2 if max_norm is None else 1)


@pytest.fixture
def host_clip(monkeypatch):
    """A PoetxGradClip on the host whose calls are recorded: (counts or None, norm, workspace,
    stream)."""
    from orthogonal_reparameterized_packed_gb300 import block
    calls = []

    def counts(n, at):
        return list((ctypes.c_int64 * n).from_address(at)) if at or not n else None

    class Library:
        def poetx_grad_norm(self, n, grads, c, types, norm, room, size, stream):
            calls.append((counts(n, c), norm, room, stream))
            return 0

        def poetx_clip_grads(self, n, grads, outs, c, types, most, norm, room, size, stream):
            calls.append((counts(n, c), norm, room, stream))
            return 0

    monkeypatch.setattr(block, "load_library", Library)
    clip = block.PoetxGradClip(device="cpu")
    clip.calls = calls
    return clip


def test_clip_takes_any_iterable_whole(host_clip):
    a, b = on_gpu(8), on_gpu(6)
    host_clip.total((t for t in (a, b)), stream=7)
    host_clip.clip((t for t in (a, b)), 1.0, stream=7)
    host_clip.clip(iter([a, b]), 1.0, out=(t for t in (a, b)), stream=7)
    assert [c[0] for c in host_clip.calls] == [[8, 6]] * 3


def test_clip_has_buffers_of_its_own_on_every_stream(host_clip):
    few, many = [on_gpu(4)], [on_gpu(4)] * 1500
    norms = [host_clip.total(few, stream=5), host_clip.clip(few, 1.0, stream=6),
             host_clip.total(many, stream=6), host_clip.clip(many, 1.0, stream=5),
             host_clip.clip(few, 1.0, stream=5)]
    _, norm, room, stream = zip(*host_clip.calls)
    assert stream == (5, 6, 6, 5, 5)
    assert norm[0] == norm[3] == norm[4] != norm[1] == norm[2]
    assert list(norm) == [t.data_ptr() for t in norms] and host_clip.norm is norms[-1]
    assert len({room[i] for i in (0, 1, 2, 3)}) == 4  # no two streams, no two sizes share one
    assert room[4] == room[3]


def test_what_a_call_needs_comes_from_its_stream(monkeypatch):
    # the stream that is current while memory is taken is the call's
    seen = []

    class Current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            seen.append(self.stream)

        def __exit__(self, *a):
            pass

    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    cuda = torch.device("cuda")
    with poetx._allocating_on(77, cuda), poetx._allocating_on("a stream", cuda):
        pass
    with poetx._allocating_on(None, cuda), poetx._allocating_on(3, torch.device("cpu")):
        pass
    assert seen == [77, "a stream"]


def test_adam_takes_its_workspace_from_the_call_s_stream(lib, monkeypatch):
    from orthogonal_reparameterized_packed_gb300 import layer
    inside, taken = [], []

    class Marked:
        def __init__(self, stream, device):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *a):
            inside.pop()

    monkeypatch.setattr(layer, "_allocating_on", Marked, raising=False)
    monkeypatch.setattr(layer, "poetx_grad_norm_workspace_size", lambda n: 64)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (taken.append(list(inside)), on_gpu(64))[1])
    layer.PoetxAdam([on_gpu(8)], lr=1e-3).step([on_gpu(8)], stream=11, max_norm=1.0)
    assert taken == [[11], [11]]


def test_outputs_over_other_inputs_are_refused(L):
    # z over the residual; q's outputs over k's inputs and the other way round; rows in place
    # at another distance.  What is allowed would be launched, and is run on a GPU elsewhere.
    f, A = ctypes.c_float, [FAKE + 65536 * i for i in range(8)]
    assert L.poetx_linear_forward(A[0], A[1], None, A[2], A[3], A[2], 64, 64, 8, 0, B, None, 0,
                                  None) == 1

    def fwd(q=A[0], k=A[1], oq=A[2], ok=A[3], loq=512):
        return L.poetx_qk_norm_rope_forward(q, k, None, None, None, None, None, oq, ok, 512, 128,
                                            loq, 128, 4, 1, 128, 0, 0, 0, f(1e-6), 3, B, None)

    def bwd(gq=A[0], gk=A[1], q=A[2], k=A[3], dq=A[4], dk=A[5], ldq=512):
        return L.poetx_qk_norm_rope_backward(gq, gk, q, k, None, None, None, None, None, dq, dk,
                                             None, None, 512, 128, 512, 128, ldq, 128, 4, 1, 128,
                                             0, 0, 0, f(1e-6), 3, B, A[7], 1 << 40, None)

    for kw in (dict(oq=A[1]), dict(ok=A[0]), dict(oq=A[0], loq=520)):
        assert fwd(**kw) == 1, kw
    for kw in (dict(dq=A[1]), dict(dq=A[3]), dict(dk=A[0]), dict(dk=A[2]),
               dict(dq=A[0], ldq=520), dict(dq=A[2], ldq=520)):
        assert bwd(**kw) == 1, kw
