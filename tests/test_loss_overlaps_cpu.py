"""What the head's losses refuse of outputs that lie over an input or over each other, in
part or whole (no GPU needed: refused before anything is enqueued)."""

import ctypes

import pytest

import orthogonal_reparameterized_packed_gb300 as poetx
from orthogonal_reparameterized_packed_gb300.build import build_library

B, F = poetx.BF16, poetx.F32
MB = 1 << 20  # between tensors; never dereferenced on these paths
D, V, T, TOP = 64, 1000, 40, 8


@pytest.fixture(scope="module")
def L():
    build_library()
    return poetx.load_library()


def addresses(es, top):
    """(start, bytes) of every tensor of a call; the workspace comes last."""
    sizes = dict(x=T * D * es, W=V * D * es, idx=T * top * 8, s=T * top * 4, w=T * 4, loss=T * 4,
                 total=4, dx=T * D * es, dW=V * D * es)
    return {k: ((i + 1) * MB, n) for i, (k, n) in enumerate(sizes.items())}


@pytest.mark.parametrize("op", ["cross entropy", "distillation"])
@pytest.mark.parametrize("code", [B, F])
def test_overlaps_are_refused(L, op, code):
    es, top = (2 if code == B else 4), (1 if op == "cross entropy" else TOP)
    at = addresses(es, top)
    size = (L.poetx_cross_entropy_workspace_size(D, V, T, code, 3, 0) if top == 1 else
            L.poetx_distill_workspace_size(D, V, T, top, code, 3, 0))

    def call(work=100 * MB, **moved):
        a = {k: moved.get(k, v[0]) for k, v in at.items()}
        if top == 1:
            return L.poetx_cross_entropy(a["x"], a["W"], a["idx"], 8, a["w"], a["loss"], a["total"],
                                         a["dx"], a["dW"], D, V, T, code, 0, work, size, None)
        return L.poetx_distill(a["x"], a["W"], a["idx"], 8, a["s"], F, a["w"], a["loss"],
                               a["total"], a["dx"], a["dW"], D, V, T, top, ctypes.c_float(2.0),
                               code, 0, work, size, None)

    inputs = ["x", "W", "idx", "w"] + (["s"] if top > 1 else [])
    outputs = ["loss", "total", "dx", "dW"]
    for o in outputs:
        for other in inputs + outputs:
            if other == o:
                continue
            start, n = at[other]
            step = 16 if o in ("dx", "dW") else 4
            places = {start, start + (n - 1) // step * step, start - at[o][1] // step * step + step}
            for p in places:  # from its start, from its last bytes on, up to its first ones
                if p < start + n and p + at[o][1] > start:
                    assert call(**{o: p}) == 1, (o, other, p - start)
    for other in inputs + outputs:  # the workspace: where a tensor lies in it
        start, n = at[other]
        for p in (start // 16 * 16, (start + n - 1) // 16 * 16, (start - size) // 16 * 16 + 16):
            if p > 0:
                assert call(work=p) == 1, (other, p - start)
