"""Cases of the operators that stand around the POET-X projections in a decoder block.

linear  z = x W^T + bias, y = act(z) + residual (W frozen), forward and backward
qk      per-head RMS norm of queries and keys with the rotary embedding, forward and backward
clip    global gradient norm over many tensors, and the clipped gradients
adam    Adam over many packed vectors with the clip applied as the gradients are read

`run` takes one pass through an operator: the plain form in elementary torch operations (float32,
rounded once at the end) or, with `own`, the library's call.  `exact` is the same in float64.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}

# Adam's hyperparameters are float32 values: the library takes them as such.
_LR, _B1, _B2, _EPS, _WD = (float(torch.tensor(v, dtype=torch.float32)) for v in
                            (1e-3, 0.9, 0.999, 1e-8, 0.01))
_STEP = 10
_CLIP_EPS = 1e-6


def listed():
    return [
        # the o projection of a merged layer for one generated token, added to the residual stream
        dict(name="linear_decode_1", op="linear", T=1, d_in=4096, d_out=4096, act="none",
             bias=False, residual=True, save_z=False, dtype="bf16"),
        # a gate projection for a batch of 24 sequences that generate one token each
        dict(name="linear_batch_24", op="linear", T=24, d_in=4096, d_out=14336, act="silu",
             bias=True, residual=False, save_z=False, dtype="bf16"),
        # the up projection of the 2048 -> 5632 layer over an odd number of prompt tokens, kept for a
        # backward pass
        dict(name="linear_prefill_2049", op="linear", T=2049, d_in=2048, d_out=5632,
             act="gelu_tanh", bias=True, residual=False, save_z=True, dtype="bf16"),
        # a training batch through the widest projection of the Llama-3-8B block
        dict(name="linear_train_8192", op="linear", T=8192, d_in=14336, d_out=4096, act="none",
             bias=True, residual=True, save_z=False, dtype="bf16"),
        # float32 layer of odd sizes with everything in the epilogue
        dict(name="linear_f32_515", op="linear", T=515, d_in=1000, d_out=777, act="gelu",
             bias=True, residual=True, save_z=True, dtype="f32"),
        # gradients of the 2048 -> 5632 projection with its activation and bias
        dict(name="linear_backward_8192", op="linear_bwd", T=8192, d_in=2048, d_out=5632,
             act="silu", dtype="bf16"),
        # one generated token of the Llama-3-8B block: 32 query and 8 key heads of 128
        dict(name="qk_decode_1", op="qk", T=1, hq=32, hk=8, D=128, rot=128, interleaved=False,
             fused=True, dtype="bf16"),
        # the bench's 16384 training tokens, q and k slices of one fused projection
        dict(name="qk_train_16384", op="qk", T=16384, hq=32, hk=8, D=128, rot=128,
             interleaved=False, fused=True, dtype="bf16"),
        # gradients at 8192 tokens
        dict(name="qk_backward_8192", op="qk_bwd", T=8192, hq=32, hk=8, D=128, rot=128,
             interleaved=False, fused=False, dtype="bf16"),
        # float32, partial rotation in interleaved pairs, heads of 80, an odd number of tokens
        dict(name="qk_backward_f32_1001", op="qk_bwd", T=1001, hq=12, hk=12, D=80, rot=32,
             interleaved=True, fused=False, dtype="f32"),
        # the packed gradients of the 14 factors of one decoder block, clipped
        dict(name="clip_block", op="clip", tensors=14, n=522240, ragged=1, gain=2.0, dtype="f32"),
        # the optimizer step of a 1.3B-shaped model's 336 packed vectors, clipped on the way
        dict(name="adam_model", op="adam", tensors=336, n=261120, ragged=7, gain=3.0, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "qk", "qk_bwd", "clip", "adam"])
    if op in ("linear", "linear_bwd"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        top = 8192 * 14336 * 4096 if dtype == "bf16" else 2048 * 2048 * 2048
        while True:
            T = _log(rng, 1, 16384)
            d_in, d_out = (_log(rng, 64, 14336) for _ in range(2))
            # feature counts of real layers are multiples of 8 nearly always; a vocabulary or a
            # float32 head need not be
            if dtype == "bf16" or rng.random() < 0.5:
                d_in -= d_in % 8
            if rng.random() < 0.7:
                d_out -= d_out % 8
            if T * d_in * d_out <= top:
                break
        c = dict(op=op, T=T, d_in=d_in, d_out=d_out, dtype=dtype,
                 act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]))
        if op == "linear":
            c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                     save_z=rng.random() < 0.4)
        return c
    if op in ("qk", "qk_bwd"):
        while True:
            T, D = _log(rng, 1, 16384), rng.choice([48, 64, 72, 80, 96, 128, 128, 192, 256])
            hk = rng.choice([1, 2, 4, 8, 12, 16])
            hq = hk * rng.choice([1, 2, 4, 8])
            if T * (hq + hk) * D <= 16384 * 40 * 128:
                break
        rot = rng.choice([D, D, D // 2])
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, rot=rot - rot % 2,
                    interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    while True:
        tensors, n = _log(rng, 1, 336), _log(rng, 1, 4000000)
        if tensors * n <= 336 * 261120:
            break
    # gains on both sides of the clip
    return dict(op=op, tensors=tensors, n=n, ragged=rng.choice([0, 1, 3, 5]),
                gain=rng.choice([0.3, 2.0, 10.0]),
                dtype="f32" if op == "adam" else rng.choice(["f32", "f32", "bf16"]))


def _counts(c):
    """Sizes of the tensors: n, and with `ragged` every other one a few elements less, so that views
    of one allocation start at odd places."""
    return [max(1, c["n"] - (c["ragged"] * i if i % 2 else 0)) for i in range(c["tensors"])]


def work(c):
    e = _ES[c["dtype"]]
    if c["op"] == "linear":
        T, a, b = c["T"], c["d_in"], c["d_out"]
        by = e * (T * a + a * b + T * b * (1 + c["residual"] + c["save_z"])) + 4 * b * c["bias"]
        return {"bytes": by, "flops": 2 * T * a * b}
    if c["op"] == "linear_bwd":
        T, a, b = c["T"], c["d_in"], c["d_out"]
        by = e * (T * a + a * b + T * b * (1 + (c["act"] != "none"))) + 4 * b
        return {"bytes": by, "flops": 2 * T * a * b}
    if c["op"] in ("qk", "qk_bwd"):
        el = c["T"] * (c["hq"] + c["hk"]) * c["D"]
        passes = 2 if c["op"] == "qk" else 3
        return {"bytes": passes * e * el + c["T"] * (4 + 4 * c["rot"]) + 8 * c["D"],
                "flops": (8 if c["op"] == "qk" else 16) * el}
    n = sum(_counts(c))
    if c["op"] == "clip":
        return {"bytes": 2 * e * n, "flops": 3 * n}
    return {"bytes": 28 * n, "flops": 16 * n}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"c": c}
    if c["op"] in ("linear", "linear_bwd"):
        T, a, b = c["T"], c["d_in"], c["d_out"]
        s["W"] = normal(b, a, scale=a ** -0.5)
        if c["op"] == "linear":
            s["x"] = normal(T, a)
            s["bias"] = normal(b, scale=0.2, dtype=torch.float32) if c["bias"] else None
            s["residual"] = normal(T, b) if c["residual"] else None
        else:
            s["dy"] = normal(T, b, scale=0.05)
            s["z"] = normal(T, b)
        if own:  # the output buffers and the workspace that a program keeps with its layer
            from orthogonal_reparameterized_packed_gb300.block import PoetxLinear
            s["layer"] = PoetxLinear(a, b, T, act=c["act"], dtype=c["dtype"],
                                     save_z=c.get("save_z", False),
                                     backward=c["op"] == "linear_bwd")
    elif c["op"] in ("qk", "qk_bwd"):
        T, hq, hk, D, rot = c["T"], c["hq"], c["hk"], c["D"], c["rot"]
        if c["fused"]:  # slices of the fused q, k, v projection's output
            qkv = normal(T, (hq + 2 * hk) * D)
            s["q"], s["k"] = qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D]
        else:
            s["q"], s["k"] = normal(T, hq * D), normal(T, hk * D)
        for n in ("gamma_q", "gamma_k"):
            s[n] = 1 + normal(D, scale=0.1, dtype=torch.float32)
        limit = T + 100
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(limit, device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = int(torch.randint(0, 100, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int32)
        if c["op"] == "qk_bwd":
            s["dq"], s["dk"] = normal(T, hq * D, scale=0.05), normal(T, hk * D, scale=0.05)
        if own:
            from orthogonal_reparameterized_packed_gb300.block import PoetxQKNormRope
            s["layer"] = PoetxQKNormRope(hq, hk, D, T, rot_dim=rot, eps=1e-6,
                                         interleaved=c["interleaved"], dtype=c["dtype"],
                                         backward=c["op"] == "qk_bwd")
    else:
        counts = _counts(c)
        n = sum(counts)
        s["grad"] = normal(n, scale=c["gain"] / math.sqrt(n))
        s["grads"] = s["grad"].split(counts)
        if c["op"] == "clip":
            s["out"] = torch.empty_like(s["grad"])
            s["outs"] = s["out"].split(counts)
        else:
            s["theta"] = normal(n, scale=0.02)
            s["m"] = normal(n, scale=0.3 * c["gain"] / math.sqrt(n))
            s["v"] = normal(n, scale=c["gain"] / math.sqrt(n)).square()
            s["thetas"], s["ms"], s["vs"] = (s[k].split(counts) for k in ("theta", "m", "v"))
        if own:
            if c["op"] == "clip":
                from orthogonal_reparameterized_packed_gb300.block import PoetxGradClip
                s["clip"] = PoetxGradClip()
            else:
                from orthogonal_reparameterized_packed_gb300.layer import PoetxAdam
                s["adam"] = PoetxAdam(s["thetas"], lr=_LR, betas=(_B1, _B2), eps=_EPS,
                                      weight_decay=_WD)
                s["adam"].m, s["adam"].v = s["ms"], s["vs"]
    return s


# ----------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + (-z).exp())
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + (-z).exp())
        return sg * (1 + z * (1 - sg))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * (-0.5 * z * z).exp() / math.sqrt(2 * math.pi))
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _plain_linear(s, c):
    z = s["x"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dt = _DT[c["dtype"]]
    return (y.to(dt), z.to(dt)) if c["save_z"] else y.to(dt)


def _plain_linear_bwd(s, c):
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _dact(s["z"].float(), c["act"])
    return (dz @ s["W"].float()).to(_DT[c["dtype"]]), dz.sum(0)


def _halves(n, rot, interleaved):
    if interleaved:
        return n[..., 0:rot:2], n[..., 1:rot:2]
    return n[..., :rot // 2], n[..., rot // 2:rot]


def _joined(a, b, rest, interleaved):
    both = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((both, rest), -1)


def _plain_head(x, h, gamma, cos, sin, c):
    x = x.float().reshape(c["T"], h, c["D"])
    n = x * (1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) * gamma
    a, b = _halves(n, c["rot"], c["interleaved"])
    y = _joined(a * cos - b * sin, b * cos + a * sin, n[..., c["rot"]:], c["interleaved"])
    return y.reshape(c["T"], -1).to(_DT[c["dtype"]])


def _plain_head_bwd(dy, x, h, gamma, cos, sin, c):
    x = x.float().reshape(c["T"], h, c["D"])
    dy = dy.float().reshape(c["T"], h, c["D"])
    r = 1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    a, b = _halves(dy, c["rot"], c["interleaved"])
    dn = _joined(a * cos + b * sin, b * cos - a * sin, dy[..., c["rot"]:], c["interleaved"])
    dg = (dn * x * r).sum((0, 1))
    gd = dn * gamma
    dx = r * (gd - x * (r * r * (gd * x).mean(-1, keepdim=True)))
    return dx.reshape(c["T"], -1).to(_DT[c["dtype"]]), dg


def _plain_scale(grads):
    norm = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
    return norm, (1.0 / (norm + _CLIP_EPS)).clamp(max=1.0)


def _plain_adam(theta, g, m, v):
    m.mul_(_B1).add_(g * (1 - _B1))
    v.mul_(_B2).add_(g * g * (1 - _B2))
    step = (m / (1 - _B1 ** _STEP)) / ((v / (1 - _B2 ** _STEP)).sqrt() + _EPS)
    theta.sub_(_LR * (step + _WD * theta))


def run(s):
    c = s["c"]
    op = c["op"]
    if own:
        return _run_own(s, c, op)
    if op == "linear":
        return _plain_linear(s, c)
    if op == "linear_bwd":
        return _plain_linear_bwd(s, c)
    if op in ("qk", "qk_bwd"):
        at = s["positions"].long()
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
        if op == "qk":
            return (_plain_head(s["q"], c["hq"], s["gamma_q"], cos, sin, c),
                    _plain_head(s["k"], c["hk"], s["gamma_k"], cos, sin, c))
        dq, dgq = _plain_head_bwd(s["dq"], s["q"], c["hq"], s["gamma_q"], cos, sin, c)
        dk, dgk = _plain_head_bwd(s["dk"], s["k"], c["hk"], s["gamma_k"], cos, sin, c)
        return dq, dk, dgq, dgk
    norm, scale = _plain_scale(s["grads"])
    if op == "clip":
        [o.copy_(g.float() * scale) for o, g in zip(s["outs"], s["grads"])]
        return norm, s["out"]
    [_plain_adam(t, g * scale, m, v)
     for t, g, m, v in zip(s["thetas"], s["grads"], s["ms"], s["vs"])]
    return norm, s["theta"], s["m"], s["v"]


def _run_own(s, c, op):
    if op == "linear":
        y = s["layer"].forward(s["x"], s["W"], s["bias"], s["residual"])
        return (y, s["layer"].z) if c["save_z"] else y
    if op == "linear_bwd":
        return s["layer"].backward(s["dy"], s["W"], z=s["z"])
    if op == "qk":
        return s["layer"].forward(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["cos"], s["sin"],
                                  s["positions"])
    if op == "qk_bwd":
        return s["layer"].backward(s["dq"], s["dk"], s["q"], s["k"], s["gamma_q"], s["gamma_k"],
                                   s["cos"], s["sin"], s["positions"])
    if op == "clip":
        norm = s["clip"].clip(s["grads"], 1.0, out=s["outs"])
        return norm, s["out"]
    s["adam"].t = _STEP - 1
    s["adam"].step(s["grads"], max_norm=1.0)
    return s["adam"].norm, s["theta"], s["m"], s["v"]


# ------------------------------------------------------- the same in 64 bits

def _exact_rows(x, h, gamma, c):
    """Rows, their root mean squares and the weights in float64."""
    x = x.double().unflatten(-1, (h, c["D"]))
    return x, ((x ** 2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt(), gamma.double()


def _exact_turn(v, angle_cos, angle_sin, c, back):
    """The rotation (or its transpose) as complex multiplication."""
    r, w = c["rot"], v.clone()
    ia = torch.arange(0, r, 2) if c["interleaved"] else torch.arange(r // 2)
    ib = ia + (1 if c["interleaved"] else r // 2)
    ia, ib = ia.to(v.device), ib.to(v.device)
    u = torch.complex(v[..., ia], v[..., ib])
    t = torch.complex(angle_cos, -angle_sin if back else angle_sin)
    u = u * t.unsqueeze(1)
    w[..., ia], w[..., ib] = u.real, u.imag
    return w


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    op = c["op"]
    if op == "linear":
        z = torch.nn.functional.linear(s["x"].double(), s["W"].double())
        if c["bias"]:
            z += s["bias"].double()
        y = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
             "gelu": lambda t: torch.nn.functional.gelu(t),
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[c["act"]](z)
        if c["residual"]:
            y = y + s["residual"].double()
        return (y, z) if c["save_z"] else y
    if op == "linear_bwd":
        dy, z = s["dy"].double(), s["z"].double()
        if c["act"] == "none":
            dz = dy
        elif c["act"] == "relu":
            dz = torch.where(z > 0, dy, torch.zeros_like(dy))
        elif c["act"] == "silu":
            sg = torch.sigmoid(z)
            dz = dy * (sg + z * sg * torch.sigmoid(-z))
        elif c["act"] == "gelu":
            dz = dy * (torch.erfc(-z / math.sqrt(2)) / 2
                       + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        else:
            a = math.sqrt(2 / math.pi)
            sg = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))  # (1 + tanh(u)) / 2
            dz = dy * (sg + z * sg * (1 - sg) * 2 * a * (1 + 0.134145 * z ** 2))
        return dz @ s["W"].double(), dz.sum(0)
    if op in ("qk", "qk_bwd"):
        at = s["positions"].long()
        cs, sn = s["cos"].double()[at], s["sin"].double()[at]
        res, grads = [], []
        for name, h, gm in (("q", c["hq"], "gamma_q"), ("k", c["hk"], "gamma_k")):
            x, rms, g = _exact_rows(s[name], h, s[gm], c)
            hat = x / rms
            if op == "qk":
                res.append(_exact_turn(hat * g, cs, sn, c, False).flatten(1))
                continue
            dn = _exact_turn(s["d" + name].double().unflatten(-1, (h, c["D"])), cs, sn, c, True)
            grads.append((dn * hat).sum(1).sum(0))
            dh = dn * g
            res.append(((dh - hat * (dh * hat).sum(-1, keepdim=True) / c["D"]) / rms).flatten(1))
        return (*res, *grads)
    grad = s["grad"].double()
    norm = torch.linalg.vector_norm(grad)
    scaled = grad * min(1.0, 1.0 / (float(norm) + _CLIP_EPS))
    if op == "clip":
        return norm, scaled
    m = _B1 * s["m"].double() + (1 - _B1) * scaled
    v = _B2 * s["v"].double() + (1 - _B2) * scaled ** 2
    theta = s["theta"].double()
    theta = theta - _LR * (m / (1 - _B1 ** _STEP) / (torch.sqrt(v / (1 - _B2 ** _STEP)) + _EPS)
                           + _WD * theta)
    return norm, theta, m, v
