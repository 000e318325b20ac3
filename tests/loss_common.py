"""What the GPU tests of the head's losses share: inputs, calls and error bounds.

Bounds.  u = 2^-8 or 2^-24 is the unit roundoff of the working type.
 logits   a sum of d fp32 products in any order, rounded to nearest or towards
          zero, is within d 2^-23 S of the exact one, S the sum of the products'
          magnitudes; divided by tau.
 terms    e^(u_v - r) for a reference r of the row: the difference is rounded (and
          the product with log2 e before it) to 2^-22 (|u_v| + |r|), the
          exponential is good to 2^-21.  |r| is at most the row's largest |u| + 64.
 sums     no term of a softmax's sum passes through more than 512 + V / 128
          additions of fp32.
 entries  the teacher's p: differences are rounded to 2^-23 of themselves, each
          exponential to 2^-21, the sum of K to K 2^-24; log p alike.
 dz       e / sum - p, each with the errors above.  bf16 rounds each difference to
          u for the products, and shifts the row's factor by the error that its
          entries' terms have in common: a weighted mean of theirs, at most u.  For
          dW x times the factor is rounded to u too; products of V (dx) or T (dW)
          terms add V or T times 2^-23 of their magnitudes; the result is rounded
          once."""

import numpy as np
import torch

from oracle import loss_oracle as lo
from tests.block_common import EPS, TDT, host, rounded


def make(T, d, V, K, dtype, seed, spread=2.0, ignored=0.0, x_scale=1.0):
    """Device tensors and the float64 values they hold."""
    rng = np.random.default_rng(seed)
    W = rounded(rng.standard_normal((V, d)) * spread / np.sqrt(d), dtype)
    idx = rng.integers(0, V, (T, K))
    x = rng.standard_normal((T, d)) + 2.0 * W[1][idx[:, 0]]
    x = rounded(x * x_scale, dtype)
    s = np.sort(rng.standard_normal((T, K)) * 2.0, 1)[:, ::-1].astype(np.float32).astype(np.float64)
    off = rng.permutation(T)[:int(round(T * ignored))]
    idx[off] = -1
    w = rng.uniform(0.1, 1.0, T).astype(np.float32).astype(np.float64)
    return dict(x=x, W=W, idx=idx, s=s, w=w, T=T, d=d, V=V, K=K, dtype=dtype)


def bounds(c, tau, weights, logits):
    """(want, bound) of loss, total, dx, dW from the oracle, as numpy arrays."""
    x, W = c["x"][1], c["W"][1]
    loss, total, dx, dW, m = lo.head_loss(x, W, c["idx"], logits, weights, tau)
    rows, w, q, P, dz, p = m["rows"], m["w"], m["q"], m["P"], m["dz"], m["p"]
    T, d, V, K = c["T"], c["d"], c["V"], c["K"]
    u16 = EPS["bf16"] if c["dtype"] == "bf16" else 0.0
    uo = EPS[c["dtype"]]
    ax, aW = np.abs(x[rows]), np.abs(W)
    ez = d * 2.0 ** -23 * (ax @ aW.T) / tau + 2.0 ** -23 * np.abs(m["u"])
    big = np.abs(m["u"]).max(1, keepdims=True) + 64 if len(rows) else np.zeros((0, 1))
    chain = (512 + V / 128) * 2.0 ** -24
    e_term = ez + 2.0 ** -22 * 2 * big + 2.0 ** -21  # relative, first order
    e_sum = (q * e_term).sum(1, keepdims=True) + chain
    e_q = 1.01 * (e_term + e_sum) + 2.0 ** -22
    # the entries' weights
    spread = np.zeros((T, 1))
    for t in rows:
        k = m["there"][t]
        spread[t] = np.ptp(logits[t, k]) / tau
    e_p = (2.0 ** -22 * spread + 2.0 ** -20 + K * 2.0 ** -23)
    b_loss = np.zeros(T)
    dP = np.zeros(P.shape)
    for n, t in enumerate(rows):
        k = np.flatnonzero(m["there"][t])
        i = c["idx"][t, k]
        np.add.at(dP[n], i, p[t, k] * e_p[t])
        size = np.abs(m["log_p"][t, k]) + np.abs(m["u"][n, i]) + big[n]
        b_loss[t] = tau ** 2 * np.sum(p[t, k] * (
            ez[n, i] + e_sum[n] + e_p[t] * (1 + size) + (8 + K) * 2.0 ** -23 * (1 + size)))
    b_total = np.sum(w * b_loss) + T ** 0.5 * 2.0 ** -22 * np.sum(w * np.abs(loss))
    scale = (w[rows] * tau)[:, None]
    tiny = 2.0 ** -109  # fp32 takes smaller dz as 0
    b_dz = np.abs(scale) * (q * e_q + dP + (q + P) * 2.0 ** -21) + tiny
    b_dx, b_dW = np.zeros((T, d)), None
    b_dx[rows] = (b_dz + np.abs(dz) * (2 * u16 + V * 2.0 ** -23) * 1.02) @ aW
    b_dx += uo * (np.abs(dx) + b_dx) + 1e-38
    b_dW = (b_dz + np.abs(dz) * (3 * u16 + T * 2.0 ** -23) * 1.03 + b_dz * 3 * u16).T @ ax
    b_dW += uo * (np.abs(dW) + b_dW) + 1e-38
    return (loss, np.float64(total), dx, dW), (b_loss, b_total, b_dx, b_dW)


def device(c, tau_case, idx_dtype=torch.int64):
    """The call's arguments behind x and W."""
    idx = torch.from_numpy(c["idx"]).to(idx_dtype).cuda()
    if not tau_case:
        return (idx[:, 0].contiguous(),)
    return idx, torch.from_numpy(c["s"]).float().cuda()


def check(got, want, bound, names=("loss", "total", "dx", "dW")):
    from tests.block_common import within
    for g, w, b, n in zip(got, want, bound, names):
        within(host(g), w, b, n)


__all__ = ["make", "bounds", "device", "check", "EPS", "TDT", "host", "rounded"]
