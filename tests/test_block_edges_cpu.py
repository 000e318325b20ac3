"""Host-side edges of the operators around the projections (no GPU needed):
what the calls and classes refuse before anything is enqueued."""

import pytest

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
