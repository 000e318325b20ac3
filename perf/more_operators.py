"""Cases of the losses at the output head, W [vocabulary][features], from the last hidden states x.

ce       softmax cross entropy with a target per token
distill  distillation from a teacher's top logits at a temperature

`run` takes one pass: the loss of every token and their weighted sum, and for a training step the
gradients of that sum by x and, where the head is trained, by W.  The plain form keeps the logits and
takes elementary torch operations (float32, rounded once at the end); with `own` it is the library's
call, which does not keep them.  `exact` is the same in float64.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_IGNORED = -100


def _case(op, T, d, V, grad, dtype="bf16", ignored=0.0, weights=False, top=1, tau=1.0):
    return dict(op=op, T=T, d=d, V=V, grad=grad, dtype=dtype, ignored=ignored, weights=weights,
                top=top, tau=tau)


def listed():
    return [
        # the loss of one token that a user asks a score for, Llama-3-8B's head
        dict(_case("ce", 1, 4096, 128256, "none"), name="ce_score_1"),
        # scores of a batch of 24 sequences, one token each, a head of 32000 x 2048
        dict(_case("ce", 24, 2048, 32000, "none"), name="ce_score_24"),
        # perplexity of a document of an odd length whose first part, the prompt, does not count
        dict(_case("ce", 2049, 2048, 50001, "none", ignored=0.3), name="ce_eval_2049"),
        # a short fine-tuning step that trains the head too
        dict(_case("ce", 64, 1024, 32000, "xw"), name="ce_train_64"),
        # a training batch of the Llama-3-8B shapes through a frozen head
        dict(_case("ce", 4096, 4096, 128256, "x"), name="ce_train_frozen_4096"),
        # the 1.3B-shaped model's training batch, head trained, padded sequences
        dict(_case("ce", 8192, 2048, 32000, "xw", ignored=0.1), name="ce_train_8192"),
        # float32, odd sizes, the caller's own weights of the tokens
        dict(_case("ce", 515, 1000, 10007, "xw", dtype="f32", weights=True), name="ce_train_f32_515"),
        # a teacher's top 16 logits against one token of the student, no gradient
        dict(_case("distill", 1, 2048, 32000, "none", top=16, tau=2.0), name="distill_score_1"),
        # a frozen head, the teacher's top 20 at temperature 1, a fifth of the tokens without any
        dict(_case("distill", 2047, 2048, 32000, "x", ignored=0.2, top=20),
             name="distill_train_frozen_2047"),
        # the largest: the top 64 of a teacher, Llama-3-8B shapes, head trained
        dict(_case("distill", 4096, 4096, 128256, "xw", top=64, tau=2.0), name="distill_train_4096"),
        # float32, odd sizes, a high temperature
        dict(_case("distill", 333, 768, 30001, "xw", dtype="f32", top=7, tau=4.0),
             name="distill_train_f32_333"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_PRODUCTS = {"none": 1, "x": 2, "xw": 3}


def draw(rng):
    op = rng.choice(["ce", "distill"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    grad = rng.choice(["none", "x", "xw", "xw"])
    # float32 is what small models and checks train in
    most = 3 * 4096 * 4096 * 128256 if dtype == "bf16" else 3 * 515 * 2048 * 32000
    while True:
        T, d, V = _log(rng, 1, 8192), _log(rng, 64, 4096), _log(rng, 300, 128256)
        # hidden sizes of real models are multiples of 8; a float32 head's need not be
        if dtype == "bf16" or rng.random() < 0.5:
            d -= d % 8
        if _PRODUCTS[grad] * T * d * V <= most:
            break
    c = _case(op, T, d, V, grad, dtype=dtype, ignored=rng.choice([0.0, 0.0, 0.1, 0.6]),
              weights=rng.random() < 0.3)
    if op == "distill":
        c.update(top=_log(rng, 1, 128), tau=rng.choice([1.0, 1.5, 2.0, 4.0]))
    return c


def _counted(c):
    return max(1, round(c["T"] * (1 - c["ignored"])))


def work(c):
    e, n, d, V = _ES[c["dtype"]], _counted(c), c["d"], c["V"]
    by = e * (n * d + V * d) + 4 * c["T"] + c["T"] * c["top"] * (8 if c["op"] == "ce" else 12)
    if c["grad"] != "none":
        by += e * c["T"] * d
    if c["grad"] == "xw":
        by += e * V * d
    return {"bytes": by, "flops": 2 * _PRODUCTS[c["grad"]] * n * d * V}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, T, d, V, K = _DT[c["dtype"]], c["T"], c["d"], c["V"], c["top"]
    s = {"c": c}
    # logits of a spread of 2, those of the right token (the teacher's likeliest) about 10 above
    s["W"] = (torch.randn((V, d), generator=g, device="cuda") * (2 * d ** -0.5)).to(dt)
    at = torch.randint(0, V, (T, K), generator=g, device="cuda")
    x = torch.randn((T, d), generator=g, device="cuda")
    lift = torch.rand((T, 1), generator=g, device="cuda") * 4 + 3
    s["x"] = (x + lift * 0.5 * s["W"][at[:, 0]].float()).to(dt)
    off = torch.zeros((T,), dtype=torch.bool, device="cuda")
    if c["ignored"]:
        off[torch.randperm(T, generator=g, device="cuda")[:T - _counted(c)]] = True
    if c["op"] == "ce":
        s["targets"] = torch.where(off, _IGNORED, at[:, 0])
    else:
        fall = 2.0 * torch.log(torch.arange(1, K + 1, device="cuda", dtype=torch.float32))
        noise = torch.randn((T, K), generator=g, device="cuda") * 0.5
        s["top_logits"] = (12.0 - fall + noise).sort(1, descending=True).values
        s["top_indices"] = torch.where(off[:, None], -1, at)
    s["weights"] = None
    if c["weights"]:
        s["weights"] = torch.rand((T,), generator=g, device="cuda") / T
    if own:  # the output buffers and the workspace that a program keeps with its head
        from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
        kw = dict(dtype=c["dtype"], backward=c["grad"] != "none", weight_grad=c["grad"] == "xw")
        if c["op"] == "ce":
            s["head"] = PoetxCrossEntropy(d, V, T, **kw)
        else:
            s["head"] = PoetxDistill(d, V, T, top=K, temperature=c["tau"], **kw)
    return s


# ----------------------------------------------------------------- plain forms

def _plain(s, c):
    dt, tau = _DT[c["dtype"]], c["tau"]
    x, W = s["x"].float(), s["W"].float()
    if c["op"] == "ce":
        idx, have = s["targets"][:, None], (s["targets"] >= 0)[:, None]
        p = have.float()
        log_p = torch.zeros_like(p)
    else:
        idx, have = s["top_indices"], s["top_indices"] >= 0
        l = torch.where(have, s["top_logits"], -math.inf)
        u = (l - l.amax(1, keepdim=True)) / tau
        u = torch.where(have, u, -math.inf)
        su = u.exp().sum(1, keepdim=True)
        log_p = torch.where(have, u - su.log(), 0.0)
        p = torch.where(have, log_p.exp(), 0.0)
    idx = idx.clamp(min=0)
    on = have.any(1)
    z = x @ W.t()
    z *= 1 / tau
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, idx)
    z -= top
    z.exp_()
    total_e = z.sum(1, keepdim=True)
    loss = tau * tau * (p * (log_p - ((picked - top) - total_e.log()))).sum(1)
    loss = torch.where(on, loss, 0.0)
    w = s["weights"] if s["weights"] is not None else 1.0 / on.sum().clamp(min=1).float()
    w = torch.where(on, w, 0.0)
    total = (w * loss).sum()
    if c["grad"] == "none":
        return loss, total
    z /= total_e
    z.scatter_add_(1, idx, -p)
    z *= (w * tau)[:, None]
    dx = (z @ W).to(dt)
    if c["grad"] == "x":
        return loss, total, dx
    return loss, total, dx, (z.t() @ x).to(dt)


def _own(s, c):
    h = s["head"]
    given = ((s["x"], s["W"], s["targets"], s["weights"]) if c["op"] == "ce" else
             (s["x"], s["W"], s["top_indices"], s["top_logits"], s["weights"]))
    if c["grad"] == "none":
        return h.forward(*given), h.total
    loss, dx, dW = h.step(*given)
    return (loss, h.total, dx) if c["grad"] == "x" else (loss, h.total, dx, dW)


def run(s):
    return _own(s, s["c"]) if own else _plain(s, s["c"])


# ------------------------------------------------------- the same in 64 bits

def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    T, V, tau = c["T"], c["V"], c["tau"]
    W = s["W"].double()
    counted = s["targets"] >= 0 if c["op"] == "ce" else (s["top_indices"] >= 0).any(1)
    if s["weights"] is not None:
        w = s["weights"].double()
    else:
        w = torch.full((T,), 1.0 / max(1, int(counted.sum())), dtype=torch.float64, device="cuda")
    loss = torch.zeros((T,), dtype=torch.float64, device="cuda")
    dx = torch.zeros((T, c["d"]), dtype=torch.float64, device="cuda")
    dW = torch.zeros_like(W) if c["grad"] == "xw" else None
    rows = torch.nonzero(counted).flatten()
    for at in rows.split(1024):  # tokens that count, some at a time
        x = s["x"][at].double()
        logq = torch.log_softmax(torch.nn.functional.linear(x, W) / tau, 1)
        if c["op"] == "ce":
            want = torch.nn.functional.one_hot(s["targets"][at], V).double()
            loss[at] = -(want * logq).sum(1)
        else:
            # no entry of a counted token is absent here; the same index twice adds up
            logp = torch.log_softmax(s["top_logits"][at].double() / tau, 1)
            inside = logq[torch.arange(len(at), device="cuda")[:, None], s["top_indices"][at]]
            loss[at] = tau ** 2 * (logp.exp() * (logp - inside)).sum(1)
            want = torch.zeros_like(logq).scatter_add(1, s["top_indices"][at], logp.exp())
        if c["grad"] == "none":
            continue
        dlogits = (logq.exp() - want) * (tau * w[at])[:, None]
        dx[at] = dlogits @ W
        if dW is not None:
            dW += dlogits.t() @ x
    out = (loss, (loss * torch.where(counted, w, torch.zeros_like(w))).sum())
    if c["grad"] == "none":
        return out
    return (*out, dx) if c["grad"] == "x" else (*out, dx, dW)
