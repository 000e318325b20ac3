"""GPU parity of the query / key norm with the rotary embedding and of its
gradients, against the float64 oracle on the rounded inputs.

Bounds, per element (u = 2^-24, D features): mean(x^2) is a sum of D fp32
terms, relative error <= (D + 2) u, so r is within (D/2 + 6) u; n, the two
products and their sum add 6 u of the terms' magnitudes.  Forward: y is within
(D/2 + 12) u (|n_a| + |n_b|), then rounded once.  Backward: dn within 3 u of
its terms, the mean within (D + 6) u of the mean of magnitudes; dx is within
(2 D + 24) u r (|g| + |x| r^2 mean|g x|) with |g| taken over the pair.
dgamma: (rows + D/2 + 12) u sum |dn x| r."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block_oracle as bo  # noqa: E402
from tests.block_common import EPS, TDT, Guarded, host, rounded, status_ok, within  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPSILON = float(np.float32(1e-6))

# (tokens, q heads, k heads, head_dim, rot_dim, interleaved)
CASES = [(1, 32, 8, 128, 128, False), (1, 1, 1, 1, 0, False), (3, 2, 1, 2, 2, True),
         (5, 3, 0, 7, 4, False), (2, 1, 1, 17, 6, True), (37, 4, 2, 64, 64, False),
         (33, 5, 3, 64, 32, True), (20, 12, 12, 80, 32, True), (9, 7, 1, 80, 80, False),
         (64, 2, 2, 96, 96, False), (11, 6, 2, 72, 36, False), (11, 6, 2, 72, 72, True),
         (130, 8, 8, 128, 128, True), (100, 9, 5, 128, 64, False), (10, 3, 3, 192, 192, False),
         (7, 3, 1, 256, 256, True), (6, 2, 2, 512, 512, False), (5, 1, 1, 511, 510, False),
         (300, 40, 10, 16, 16, False), (257, 3, 2, 48, 24, False), (1500, 4, 2, 128, 128, False),
         # tokens' heads cut into pieces that do not divide them
         (480, 48, 12, 128, 128, False), (1500, 48, 12, 128, 128, False), (112, 32, 8, 96, 48, False), (2300, 20, 28, 64, 64, True)]


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


def dcode(px, dtype):
    return px.BF16 if dtype == "bf16" else px.F32


class Case:
    """Inputs, guarded outputs, and one call each way.  `pad`: extra elements
    between rows; `shift`: elements past the aligned start of every tensor."""

    def __init__(self, px, case, dtype, seed, pad=0, shift=0, gammas=True, positions=True):
        self.px, self.dtype = px, dtype
        self.T, self.hq, self.hk, self.D, self.rot, self.il = case
        T, D = self.T, self.D
        rng = np.random.default_rng(seed)
        self.g = Guarded()
        self.t, self.h, self.ld = {}, {}, {}
        for n, heads in (("q", self.hq), ("k", self.hk), ("gq", self.hq), ("gk", self.hk)):
            v = rng.standard_normal((T, heads, D)) * (2.0 if n in "qk" else 0.2)
            dev, self.h[n] = rounded(v, dtype)
            buf = torch.zeros((T, heads * D + pad + (pad and 8)), dtype=TDT[dtype], device="cuda")
            wide = torch.zeros((buf.numel() + shift,), dtype=TDT[dtype], device="cuda")
            rows = wide[shift:].view(buf.shape)
            rows[:, :heads * D] = dev.view(T, heads * D)
            self.t[n], self.ld[n] = rows, rows.shape[1]
        for n, heads in (("oq", self.hq), ("ok", self.hk)):
            self.ld[n] = heads * D + pad
            self.t[n] = self.g.tensor((T, self.ld[n]), TDT[dtype], shift)
        self.gam = {}
        for n in ("q", "k"):
            self.gam[n] = rounded(1 + 0.2 * rng.standard_normal(D), "f32") if gammas else (
                None, np.ones(D))
        self.rows = T + 5
        ang = rng.standard_normal((self.rows, self.rot // 2)) * 3
        self.cos, self.cos64 = rounded(np.cos(ang), "f32")
        self.sin, self.sin64 = rounded(np.sin(ang), "f32")
        self.pos64 = rng.integers(0, self.rows, T) if positions else np.arange(T)
        self.pos = torch.from_numpy(self.pos64.astype(np.int32)).cuda() if positions else None

    def k_or_none(self, name):
        return self.t[name] if self.hk else None

    def forward(self, stream=None):
        t, ld = self.t, self.ld
        self.px.poetx_qk_norm_rope_forward(
            t["q"], self.k_or_none("k"), self.gam["q"][0], self.gam["k"][0], self.cos, self.sin,
            self.pos, t["oq"], self.k_or_none("ok"), ld["q"], ld["k"], ld["oq"], ld["ok"], self.hq,
            self.hk, self.D, self.rot, self.rows, self.il, EPSILON, self.T,
            dcode(self.px, self.dtype), stream)

    def backward(self, dgammas=True, stream=None):
        t, ld, px = self.t, self.ld, self.px
        need = px.poetx_qk_norm_rope_backward_workspace_size(self.hq, self.hk, self.D, self.T,
                                                             dcode(px, self.dtype))
        ws = self.g.tensor((max(16, need),), torch.uint8)
        self.dg = [self.g.tensor((self.D,), torch.float32) if dgammas else None for _ in "qk"]
        px.poetx_qk_norm_rope_backward(
            t["gq"], self.k_or_none("gk"), t["q"], self.k_or_none("k"), self.gam["q"][0],
            self.gam["k"][0], self.cos, self.sin, self.pos, t["oq"], self.k_or_none("ok"),
            *self.dg, ld["gq"], ld["gk"], ld["q"], ld["k"], ld["oq"], ld["ok"], self.hq, self.hk,
            self.D, self.rot, self.rows, self.il, EPSILON, self.T, dcode(px, self.dtype), ws,
            stream)

    def out(self, n):
        heads = self.hq if n == "q" else self.hk
        return host(self.t["o" + n])[:, :heads * self.D].reshape(self.T, heads, self.D)

    def sides(self):
        return ["q"] + (["k"] if self.hk else [])

    def trig(self):
        return self.cos64[self.pos64], self.sin64[self.pos64]


def pair_sum(m, rot, interleaved):
    """|m_a| + |m_b| at both places of a pair."""
    a, b = bo._pairs(rot, interleaved)
    s = np.abs(m).copy()
    s[..., a] = s[..., b] = np.abs(m[..., a]) + np.abs(m[..., b])
    return s


def check_forward(c):
    status_ok(c.px)
    c.g.check()
    cos, sin = c.trig()
    for n in c.sides():
        x, gam = c.h[n], c.gam[n][1]
        want = bo.norm_rope(x, gam, cos, sin, EPSILON, c.il)
        norm = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPSILON) * gam
        b = (c.D / 2 + 12) * U * pair_sum(norm, c.rot, c.il)
        within(c.out(n), want, b + EPS[c.dtype] * (np.abs(want) + b), n)


def check_backward(c, dgammas=True):
    status_ok(c.px)
    c.g.check()
    cos, sin = c.trig()
    for i, n in enumerate(c.sides()):
        x, dy, gam = c.h[n], c.h["g" + n], c.gam[n][1]
        dx, dgam = bo.norm_rope_backward(dy, x, gam, cos, sin, EPSILON, c.il)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPSILON)
        dn = pair_sum(dy, c.rot, c.il)
        g = dn * np.abs(gam)
        b = (2 * c.D + 24) * U * r * (g + np.abs(x) * r * r * np.mean(g * np.abs(x), -1,
                                                                     keepdims=True))
        within(c.out(n), dx, b + EPS[c.dtype] * (np.abs(dx) + b), "d" + n)
        if dgammas:
            rows = x.shape[0] * x.shape[1]
            bg = (rows + c.D / 2 + 12) * U * (dn * np.abs(x) * r).sum((0, 1))
            within(host(c.dg[i]), dgam, bg, "dgamma_" + n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward_matches_oracle(px, i, dtype):
    c = Case(px, CASES[i], dtype, 200 + i, gammas=i % 5 != 4, positions=i % 3 != 2)
    c.forward()
    check_forward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward_matches_oracle(px, i, dtype):
    c = Case(px, CASES[i], dtype, 230 + i, gammas=i % 5 != 3, positions=i % 3 != 1)
    c.backward(dgammas=i % 4 != 3)
    check_backward(c, dgammas=i % 4 != 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (0, 1), (3, 0), (4, 4), (1, 3), (8, 2)])
def test_strides_and_alignments(px, pad, shift, dtype):
    for case in ((19, 4, 2, 128, 128, False), (19, 4, 2, 64, 32, True)):
        c = Case(px, case, dtype, 260, pad=pad, shift=shift)
        c.forward()
        check_forward(c)
        c = Case(px, case, dtype, 261, pad=pad, shift=shift)
        c.backward()
        check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(50, 4, 2, 128, 128, False), (50, 3, 1, 18, 10, True)])
def test_positions_outside_the_table(px, case, dtype):
    c = Case(px, case, dtype, 270)
    bad = {0: -1, 7: c.rows, 49: 2 ** 31 - 1}
    for t, p in bad.items():
        c.pos[t] = p
    keep = [t for t in range(c.T) if t not in bad]
    c.forward()
    torch.cuda.synchronize()
    assert px.poetx_device_status() == 1  # POETX_ERR_INVALID_ARG, recorded once
    c.g.check()
    cos, sin = c.cos64[c.pos64], c.sin64[c.pos64]
    for n in "qk":
        got = c.out(n)
        assert np.all(got[list(bad)] == 0)
        want = bo.norm_rope(c.h[n][keep], c.gam[n][1], cos[keep], sin[keep], EPSILON, c.il)
        scale = np.abs(want).max()
        within(got[keep], want, (EPS[dtype] + 1e-4) * scale)
    c.backward()
    torch.cuda.synchronize()
    assert px.poetx_device_status() == 1
    for i, n in enumerate("qk"):
        assert np.all(c.out(n)[list(bad)] == 0)
        _, dgam = bo.norm_rope_backward(c.h["g" + n][keep], c.h[n][keep], c.gam[n][1], cos[keep],
                                        sin[keep], EPSILON, c.il)
        within(host(c.dg[i]), dgam, 1e-4 * np.abs(c.h["g" + n] * c.h[n]).sum((0, 1)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(px, dtype):
    for case in ((30, 4, 2, 128, 128, False), (30, 2, 1, 21, 10, True)):
        a = Case(px, case, dtype, 280)
        a.forward()
        b = Case(px, case, dtype, 280)
        b.t["oq"], b.t["ok"] = b.t["q"], b.t["k"]
        b.forward()
        status_ok(px)
        assert torch.equal(a.t["oq"], b.t["q"]) and torch.equal(a.t["ok"], b.t["k"])
        a = Case(px, case, dtype, 281)
        a.backward()
        b = Case(px, case, dtype, 281)
        b.t["oq"], b.t["ok"] = b.t["gq"], b.t["gk"]
        b.backward()
        status_ok(px)
        assert torch.equal(a.t["oq"], b.t["gq"]) and torch.equal(a.t["ok"], b.t["gk"])


def test_no_tokens(px):
    z = torch.zeros((1,), device="cuda")
    dg = torch.full((2, 64), 3.0, device="cuda")
    ws = torch.empty((max(16, px.poetx_qk_norm_rope_backward_workspace_size(2, 1, 64, 0,
                                                                            px.F32)),),
                     dtype=torch.uint8, device="cuda")
    px.poetx_qk_norm_rope_forward(z, z, None, None, z, z, None, z, z, 0, 0, 0, 0, 2, 1, 64, 64, 1,
                                  False, 1e-6, 0, px.F32)
    px.poetx_qk_norm_rope_backward(z, z, z, z, None, None, z, z, None, z, z, dg[0], dg[1], 0, 0, 0,
                                   0, 0, 0, 2, 1, 64, 64, 1, False, 1e-6, 0, px.F32, ws)
    status_ok(px)
    assert torch.count_nonzero(dg) == 0


def test_rows_of_zeros_and_extreme_values(px):
    # a zero row stays zero; rows of 1e18 and 1e-18 (squares inside fp32's range) stay finite
    D = 128
    x = torch.zeros((4, D), device="cuda")
    x[1] = 1e18
    x[2] = 1e-18
    x[3, 0] = float("nan")
    from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope, rope_tables
    step = PoetxQKNormRope(1, 0, D, 4, dtype="f32")
    cos, sin = rope_tables(4, D)
    y, _ = step.forward(x, x[:, :0], None, None, cos, sin)
    status_ok(px)
    assert torch.count_nonzero(y[0]) == 0
    assert torch.isfinite(y[:3]).all() and torch.isnan(y[3]).all()
    assert abs(float(y[1].norm()) - D ** 0.5) < 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_on_another_stream_and_in_a_graph(px, dtype):
    c = Case(px, (700, 8, 2, 128, 128, False), dtype, 290)
    c.backward()
    want = [t.clone() for t in (c.t["oq"], c.t["ok"], *c.dg)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.backward(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (c.t["oq"], c.t["ok"], *c.dg)))
    from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope
    step = PoetxQKNormRope(8, 2, 128, 700, dtype=dtype, eps=EPSILON, backward=True)

    def call():
        return step.backward(c.t["gq"], c.t["gk"], c.t["q"], c.t["k"], c.gam["q"][0],
                             c.gam["k"][0], c.cos, c.sin, c.pos)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    status_ok(px)
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_class_takes_slices_and_refuses_other_layouts(px):
    from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope, rope_tables
    T, hq, hk, D = 6, 4, 2, 64
    qkv = torch.randn((T, (hq + 2 * hk) * D), device="cuda").bfloat16()
    cos, sin = rope_tables(10, D)
    step = PoetxQKNormRope(hq, hk, D, 10)
    q, k = qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D]
    a = [t.clone() for t in step.forward(q, k, None, None, cos, sin)]
    assert a[0].shape == (T, hq * D) and a[1].shape == (T, hk * D)
    b = step.forward(q.contiguous().view(T, hq, D), k.contiguous(), None, None, cos, sin)
    assert all(torch.equal(p, r) for p, r in zip(a, b))
    with pytest.raises(ValueError):
        step.forward(q.t().contiguous().t(), k, None, None, cos, sin)
    with pytest.raises(ValueError):
        step.forward(q.float(), k, None, None, cos, sin)
    with pytest.raises(ValueError):
        step.forward(q, k, None, None, cos[:, :3].contiguous(), sin)
    with pytest.raises(RuntimeError):
        step.backward(q, k, q, k, None, None, cos, sin)
