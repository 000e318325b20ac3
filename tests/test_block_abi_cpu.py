"""Host-side checks of the calls around the projections (no GPU needed):
workspace sizes, and arguments rejected before anything is enqueued."""

import ctypes

import pytest

import orthogonal_reparameterized_packed_gb300 as poetx
from orthogonal_reparameterized_packed_gb300.build import build_library

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
B, F = poetx.BF16, poetx.F32
f = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    build_library()
    return poetx.load_library()


def test_linear_rejects_invalid_arguments(L):
    ws = poetx.poetx_linear_forward_workspace_size(64, 128, 40, B)

    def fwd(x=FAKE, W=FAKE, bias=FAKE, res=FAKE, y=FAKE + 4096, z=None, d_in=64, d_out=128, T=40,
            act=0, dt=B, work=FAKE, n=1 << 40):
        return L.poetx_linear_forward(x, W, bias, res, y, z, d_in, d_out, T, act, dt, work, n,
                                      None)

    bad = [dict(x=None), dict(W=None), dict(y=None), dict(x=FAKE + 2), dict(bias=FAKE + 4),
           dict(res=FAKE + 8), dict(y=FAKE + 4100), dict(z=FAKE + 4098), dict(d_in=0),
           dict(d_out=-1), dict(T=-1), dict(T=(1 << 22) + 1), dict(act=5), dict(act=-1),
           dict(dt=2), dict(d_in=(1 << 20) + 1), dict(y=FAKE), dict(z=FAKE + 4096)]
    for kw in bad:
        assert fwd(**kw) == 1, kw
    if ws:
        assert fwd(n=ws - 1) == 3 and fwd(work=None) == 3 and fwd(work=FAKE + 8) == 3
    assert fwd(T=0, x=None, y=None, work=None, n=0) == 0

    def bwd(dy=FAKE, z=FAKE + 64, W=FAKE, dx=FAKE + 4096, db=FAKE, d_in=64, d_out=128, T=40,
            act=2, dt=B, work=FAKE, n=1 << 40):
        return L.poetx_linear_backward(dy, z, W, dx, db, d_in, d_out, T, act, dt, work, n, None)

    bad = [dict(dy=None), dict(z=None), dict(W=None), dict(dy=FAKE + 2), dict(db=FAKE + 4),
           dict(dx=FAKE), dict(dx=FAKE + 64), dict(d_in=0), dict(act=9), dict(dt=3), dict(T=-2)]
    for kw in bad:
        assert bwd(**kw) == 1, kw
    assert bwd(dx=None, db=None) == 0  # nothing wanted
    need = poetx.poetx_linear_backward_workspace_size(64, 128, 40, 2, B, True)
    assert need > 0 and bwd(n=need - 1) == 3
    assert bwd(T=0, db=None, dy=None, z=None, dx=None) == 0


def test_linear_workspace_of_invalid_sizes_is_zero():
    assert poetx.poetx_linear_forward_workspace_size(0, 64, 8, B) == 0
    assert poetx.poetx_linear_forward_workspace_size(64, 64, -1, B) == 0
    assert poetx.poetx_linear_forward_workspace_size(64, 64, 8, 7) == 0
    assert poetx.poetx_linear_backward_workspace_size(64, 64, 8, 11, B) == 0
    assert poetx.poetx_linear_backward_workspace_size(64, 64, 0, 1, B) == 0


def test_qk_norm_rope_rejects_invalid_arguments(L):
    def fwd(q=FAKE, k=FAKE, gq=FAKE, gk=FAKE, cos=FAKE, sin=FAKE, pos=FAKE, oq=FAKE, ok=FAKE,
            lq=512, lk=128, loq=512, lok=128, hq=4, hk=1, D=128, rot=128, rows=10, eps=1e-6, T=3,
            dt=B):
        return L.poetx_qk_norm_rope_forward(q, k, gq, gk, cos, sin, pos, oq, ok, lq, lk, loq, lok,
                                            hq, hk, D, rot, rows, 0, f(eps), T, dt, None)

    bad = [dict(q=None), dict(k=None), dict(oq=None), dict(ok=None), dict(q=FAKE + 1),
           dict(gq=FAKE + 2), dict(cos=None), dict(sin=None), dict(cos=FAKE + 2),
           dict(pos=FAKE + 2), dict(lq=511), dict(lk=127), dict(loq=0), dict(lok=-1), dict(hq=0),
           dict(hk=-1), dict(D=0), dict(rot=127), dict(rot=130), dict(rot=-2), dict(rows=-1),
           dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(T=-1), dict(T=(1 << 22) + 1), dict(dt=5)]
    for kw in bad:
        assert fwd(**kw) == 1, kw
    assert fwd(D=514, rot=0, lq=4 * 514, lk=514, loq=4 * 514, lok=514) == 2
    assert fwd(T=0, q=None, k=None, oq=None, ok=None) == 0

    def bwd(gq=FAKE, gk=FAKE, q=FAKE, k=FAKE, dq=FAKE, dk=FAKE, dgq=FAKE, ld=512, D=128, T=3,
            work=FAKE, n=1 << 40, cos=FAKE):
        return L.poetx_qk_norm_rope_backward(gq, gk, q, k, None, None, cos, FAKE, None, dq, dk,
                                             dgq, None, ld, 128, 512, 128, 512, 128, 4, 1, D, 128,
                                             10, 0, f(1e-6), T, B, work, n, None)

    for kw in [dict(gq=None), dict(gk=None), dict(q=None), dict(k=None), dict(dq=None),
               dict(dk=None), dict(dgq=FAKE + 1), dict(ld=500), dict(T=-1), dict(cos=None)]:
        assert bwd(**kw) == 1, kw
    need = poetx.poetx_qk_norm_rope_backward_workspace_size(4, 1, 128, 3, B)
    assert need > 0 and bwd(n=need - 1) == 3 and bwd(work=None) == 3
    assert poetx.poetx_qk_norm_rope_backward_workspace_size(4, 1, 513, 3, B) == 0


def test_lists_reject_invalid_arguments(L):
    def arr(*v):
        return (ctypes.c_void_p * len(v))(*v)

    def cnt(*v):
        return (ctypes.c_int64 * len(v))(*v)

    def types(*v):
        return (ctypes.c_int32 * len(v))(*v)

    ws = poetx.poetx_grad_norm_workspace_size(2)
    assert ws > 0 and poetx.poetx_grad_norm_workspace_size(-1) == 0
    two, c2 = arr(FAKE, FAKE), cnt(4, 4)

    def norm(n=2, g=two, c=c2, t=None, out=FAKE, work=FAKE, size=ws):
        return L.poetx_grad_norm(n, g, c, t, out, work, size, None)

    for kw in [dict(n=-1), dict(g=None), dict(c=None), dict(c=cnt(4, -1)),
               dict(c=cnt(4, (1 << 42) + 1)), dict(c=cnt(1 << 42, 1 << 42)), dict(g=arr(FAKE, 0)),
               dict(g=arr(FAKE, FAKE + 2)), dict(t=types(0, 2)), dict(out=None),
               dict(out=FAKE + 2), dict(g=arr(FAKE, FAKE + 1), t=types(1, 1))]:
        assert norm(**kw) == 1, kw
    assert norm(size=ws - 1) == 3 and norm(work=None) == 3

    def clip(o=two, mx=1.0, g=two, out=FAKE, size=ws):
        return L.poetx_clip_grads(2, g, o, c2, None, f(mx), out, FAKE, size, None)

    for kw in [dict(o=None), dict(o=arr(FAKE, 0)), dict(mx=-1.0), dict(mx=float("nan")),
               dict(g=None), dict(out=None)]:
        assert clip(**kw) == 1, kw
    assert clip(size=ws - 1) == 3

    def adam(th=two, g=two, m=two, v=two, step=1, b1=0.9, b2=0.999, eps=1e-8, mx=1.0, out=FAKE,
             work=FAKE, c=c2):
        return L.poetx_adam_update_many(2, th, g, m, v, c, step, f(1e-3), f(b1), f(b2), f(eps),
                                        f(0.0), f(mx), out, work, ws, None)

    for kw in [dict(th=None), dict(g=arr(0, FAKE)), dict(m=None), dict(v=arr(FAKE, FAKE + 2)),
               dict(step=0), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0), dict(mx=float("nan")),
               dict(out=None)]:
        assert adam(**kw) == 1, kw
    assert adam(work=None) == 3
    assert adam(c=cnt(0, 0), th=arr(0, 0), g=arr(0, 0), m=arr(0, 0), v=arr(0, 0), mx=-1.0,
                out=None, work=None) == 0  # nothing to do
