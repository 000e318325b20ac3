"""What the GPU tests of the operators around the projections share."""

import numpy as np
import torch

GUARD = 4096  # bytes on each side of an output
PATTERN = 0xA5
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # unit roundoffs: 24 and 8 significant bits
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Guarded:
    """Device buffers between guard bands that no kernel may write."""

    def __init__(self):
        self.bufs = []

    def tensor(self, shape, dtype, shift=0):
        """`shift`: elements past the aligned start."""
        es = torch.tensor([], dtype=dtype).element_size()
        nbytes = int(np.prod(shape)) * es
        raw = torch.full((2 * GUARD + nbytes + shift * es,), PATTERN, dtype=torch.uint8,
                         device="cuda")
        lo = GUARD + shift * es
        self.bufs.append((raw, lo, lo + nbytes))
        return raw[lo:lo + nbytes].view(dtype).view(*shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (raw, lo, hi) in enumerate(self.bufs):
            assert bool((raw[:lo] == PATTERN).all()), f"buffer {i}: write before its start"
            assert bool((raw[hi:] == PATTERN).all()), f"buffer {i}: write past its end"


def rounded(a, dtype):
    """(device tensor of the type, the float64 values it holds)"""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TDT[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def status_ok(px):
    torch.cuda.synchronize()
    st = px.poetx_device_status()
    assert st == 0, px.poetx_status_string(st)


def within(got, want, bound, what=""):
    """|got - want| <= bound elementwise (bound may be an array)."""
    off = np.abs(got - want) - bound
    assert np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(off), off.shape) if off.ndim else ()
    assert np.all(off <= 0), (what, worst, got[worst], want[worst],
                              np.broadcast_to(bound, off.shape)[worst])
